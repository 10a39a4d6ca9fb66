// decode.cu -- the whole layer for up to 8 tokens, from hidden states, in two kernels.
//
//   l[t][e] = <x_t, r_e> (+ b_e);  ids = the k largest, ties to the lower id
//   g[t][j] = exp(l_j - l_max) / sum over the chosen
//   h[t][j] = silu(W1_e x_t) * (W3_e x_t);  out[t] = sum_j g[t][j] W2_e h[t][j]
//
// Kernel 1 (router_kernel) is the router's product: one CTA an expert, its row
// read once for all tokens. Kernel 2 (decode_kernel) does the rest. Every CTA
// takes the top-k of the few logits itself, which costs less than a kernel or a
// wait between CTAs, and finds the chosen experts (at most T * topk) with their
// tokens. Then the work of W13, and after it that of W2, is cut into one
// share per SM of equal cost: a run of units, 32 weight rows of one expert over
// the whole K, in the order (expert, rows). Shares are claimed from a counter,
// every W13 share before any W2 share. W2 shares wait for the W13 units of
// their experts, and CTAs that find no share left for all of W2: every wait is
// for CTAs that run, whatever runs beside this kernel, and bounded.
//
// A share's steps (one or two k-blocks of a unit) are cut evenly among the CTA's
// warps, wherever in K that falls. A warp copies its steps' packed bytes into a
// ring of its own with asynchronous 16-byte copies, some k-blocks ahead and
// across unit borders, decodes them into MMA operands and issues m16n8k16 MMAs
// with the tokens as the N side; the activations are in shared memory, laid
// out as the MMAs' fragments. Warps do not wait for one another within a
// share; afterwards the warp that ends a unit adds the sums of those that
// began it, in the order of K. Every thread finds the borders of some shares at
// the start and every warp its own part of a share, so that nothing waits for a
// plan between W13 and W2 (a warp that planned each share for all: 21.1 us where
// this takes 20.6, one token of 128 experts). When all W2 units are done, each
// CTA adds the slots of an even part of the output by their gates. (Left to the
// CTA that completes a tile of 128 output rows, that falls to the few with the
// last expert, which then took 20 us more than the others for 8 tokens of 6144.)
//
// What bounds it. With one or two tokens an expert the MMAs use a quarter of
// their columns at most, so decoding the codes costs more than their bytes: a
// k-block of 16 rows takes about 40 clocks an SM, of which the copies and the
// loop alone are 26, and the bytes at the copy rate 13 (NF3). 152 SMs at that
// pace stream 3.9 TB/s (8 tokens of 256 experts, 6144 x 2048, top-8: 245 us,
// 968.6 MB; the bytes alone would take 143 us). In 4 tokens of 16 experts, 12 of
// them NF3, the ALU is 49% busy, issue 57%, shared memory 37%: the warps wait
// on each other's pipes and on their own chains. More warps (20, 24, 32), deeper rings, L2 prefetch ahead of them,
// codes loaded into registers without a ring (355 us, its waits at every use)
// and one bulk copy a warp and step (379) were all slower or equal. A
// small call is bounded by its chain of waits instead, about 13 us of logits,
// top-k, the plan, first copies, W13's counts and cold instruction fetches
// (one token of 128 experts, 2048 x 768, top-8: 20.6 us, 21.8 MB).
//
// Rounding. h stays fp32 between the products and enters W2 as the sum of two
// values of the activation type (hi + lo, 16 significant bits in bf16, 22 in
// fp16), which are two columns of the N side: with the one or two tokens that
// an expert usually has they cost nothing. One value would add its rounding's
// error to the result, as large as the result's own. In fp16 a token's h is
// brought into the type's range by a power of two first (of its largest |h|).
// NF3 scales are applied to fp32 sums of raw codebook values, NVFP4 and MXFP4
// products are exact; sums are fp32, each in one fixed order.
#include <climits>
#include <type_traits>

#include "act.cuh"
#include "common.cuh"
#include "internal.h"
#include "topk.cuh"

namespace hmoe {

// 16 warps keep the pipes busy (8 tokens of the 256-expert layer: 265 us, with 8 warps 306). Where a CTA has few steps
// of W13 (of two k-blocks) the barriers of fewer warps and their longer parts count more: 40 steps take 22.3 us with 16
// warps and 20.7 with 8, 81 steps 29.4 and 28.4, 121 steps 33.3 and 32.7, 162 steps 35.4 and 35.9, 323 steps 51.7 and
// 53.3. The rule counts every slot as an expert of its own, which the host knows.
constexpr int DK_WARPS = 16;
constexpr int DK_FEW_WARPS = 8;
constexpr int DK_FEW_STEPS = 140;  // at most
constexpr int DK_UNIT = 32;      // weight rows of a unit: two row groups of a tile
// K-blocks of a warp's ring: with 16 warps 4 keep as much in flight as the loop uses, and leave room for more activations
// (8 tokens of the 128-expert layer in fp16: 53.8 us, 55.0 with 6).
__host__ __device__ constexpr int dk_ring(int warps) { return warps == DK_FEW_WARPS ? 6 : 4; }
constexpr int DK_SLOT = 1152;    // bytes of a ring slot: a unit's k-block in the widest format
constexpr int DK_MAX_SLOTS = DECODE_MAX_TOKENS * MAX_TOPK;
// Of a slot's four NF3 words three go through a pair table and one through byte permutes, each of which loads one pipe (two
// and four words measured the same within 1%). The table (common.cuh) is indexed by the code words' bytes as they are: bits
// 3 and 7, which belong to other codes, make no difference to the entry. That saves a mask a word (one token of the
// 256-expert layer: 51.3 -> 50.8 us, 8 tokens: 250 -> 248).
constexpr int DK_NF3_ENTRIES = 256;

// Relative time of a unit's k-block, by format and type: what bounds the warps is their instructions, not the bytes
// (layers of one format and of this one shape, 2 and 4 tokens, 6144 x 2048: NF3 40, NVFP4 42, in fp16 47, MXFP4 47 to 49 clocks an SM for 16
// rows x 64 K, where the bytes are as 13 : 18 : 17). Shares by bytes took 285 us where these take 261 (8 tokens of the
// 256-expert layer, bf16), 167 where they take 156 (4 tokens, MXFP4, fp16).
template <int FMT, int ACT>
constexpr int UNIT_COST = FMT == FMT_NF3 ? 20 : (FMT == FMT_NVFP4 ? (ACT == ACT_F16 ? 23 : 21) : 24);
template <int KEPT, int ACT>
__device__ __forceinline__ int unit_cost(int fmt) {
  return fmt == FMT_NF3 ? UNIT_COST<FMT_NF3, ACT> : UNIT_COST<KEPT, ACT>;
}
template <int KEPT, int ACT>
__device__ __forceinline__ int by_unit_cost(int v, int fmt) {
  return fmt == FMT_NF3 ? v / UNIT_COST<FMT_NF3, ACT> : v / UNIT_COST<KEPT, ACT>;
}

// ------------------------------------------------------------ kernel 1: router logits
constexpr int RK_THREADS = 128;
// One CTA an expert: logits[t][e] for T <= TM tokens. fp32 sums in a fixed
// order (a thread's own values, the warp's tree, the warps in turn). Inputs that
// the kernel before may still write when this one starts are read by coherent
// loads: those of the read-only path are for what nobody writes meanwhile.
template <int ACT, int TM>
__global__ void __launch_bounds__(RK_THREADS) router_kernel(const uint16_t* __restrict__ x, const uint16_t* __restrict__ router,
                                                            const float* __restrict__ bias, int T, int H, int E,
                                                            float* __restrict__ logits) {
  __shared__ float s_part[RK_THREADS / 32][TM];
  const int e = blockIdx.x, tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  // The row to L2 while the kernel before still runs; nothing is read before the wait.
  for (int c = tid * 64; c < H; c += RK_THREADS * 64)
    asm volatile("prefetch.global.L2 [%0];" ::"l"(router + (size_t)e * H + c));
  pdl_wait();
  pdl_trigger();
  float acc[TM];
#pragma unroll
  for (int t = 0; t < TM; ++t) acc[t] = 0.0f;
  const uint16_t* row = router + (size_t)e * H;
#pragma unroll 2
  for (int c = tid * 8; c < H; c += RK_THREADS * 8) {
    const uint4 w = __ldca(reinterpret_cast<const uint4*>(row + c));
    uint4 v[TM];
#pragma unroll
    for (int t = 0; t < TM; ++t)
      v[t] = t < T ? __ldca(reinterpret_cast<const uint4*>(x + (size_t)t * H + c)) : make_uint4(0, 0, 0, 0);
    const uint32_t ww[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float2 a = act_x2_to_f32<ACT>(ww[i]);
#pragma unroll
      for (int t = 0; t < TM; ++t) {
        const uint32_t vv[4] = {v[t].x, v[t].y, v[t].z, v[t].w};
        const float2 b = act_x2_to_f32<ACT>(vv[i]);
        acc[t] = fmaf(a.x, b.x, acc[t]);
        acc[t] = fmaf(a.y, b.y, acc[t]);
      }
    }
  }
#pragma unroll
  for (int t = 0; t < TM; ++t) {
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) acc[t] += __shfl_xor_sync(0xffffffffu, acc[t], off);
    if (lane == 0) s_part[warp][t] = acc[t];
  }
  __syncthreads();
  if (tid < T) {
    float s = 0.0f;
#pragma unroll
    for (int w = 0; w < RK_THREADS / 32; ++w) s += s_part[w][tid];
    if (bias) s += __ldca(bias + e);
    logits[(size_t)tid * E + e] = isnan(s) ? __int_as_float(0x7FFFFFFF) : s;  // one NaN, which the top-k takes as the largest
  }
}

// ------------------------------------------------------------ kernel 2
// warp_route_token (topk.cuh), the same choice and gates, for few tokens, where its time counts: a lane keeps the two
// best of its logits and looks at all of them again only after it has given both, which few of k rounds need.
__device__ __forceinline__ void warp_route_few(const float* __restrict__ row, int E, int k, int lane, int* my_id,
                                               float* my_gate) {
  const int per = (E + 31) >> 5;
  uint32_t key[MAX_E / 32];
#pragma unroll
  for (int j = 0; j < MAX_E / 32; ++j) key[j] = j < per && lane + 32 * j < E ? route_key(__ldcg(row + lane + 32 * j)) : 0u;
  uint32_t taken = 0, k1 = 0, k2 = 0;
  int j1 = 0, j2 = 0;
  auto scan = [&]() {  // j ascending: the first of equal keys has the lowest id
    k1 = k2 = 0;
    j1 = j2 = 0;
#pragma unroll
    for (int j = 0; j < MAX_E / 32; ++j) {
      if (j >= per) break;
      const uint32_t v = (taken >> j) & 1u ? 0u : key[j];
      if (v > k1) {
        k2 = k1;
        j2 = j1;
        k1 = v;
        j1 = j;
      } else if (v > k2) {
        k2 = v;
        j2 = j;
      }
    }
  };
  bool spent = true;
  int rid = 0;
  uint32_t rkey = 0;
  for (int r = 0; r < k; ++r) {
    if (__any_sync(0xffffffffu, spent)) {
      if (spent) scan();
      spent = false;
    }
    const uint32_t m = __reduce_max_sync(0xffffffffu, k1);
    const uint32_t w = __reduce_min_sync(0xffffffffu, k1 == m ? (uint32_t)(lane + 32 * j1) : 0xFFFFFFFFu);
    if ((int)(w & 31u) == lane) {
      taken |= 1u << (w >> 5);
      k1 = k2;
      j1 = j2;
      spent = k2 == 0u;
      k2 = 0u;
    }
    if (lane == r) {
      rid = (int)w;
      rkey = m;
    }
  }
  const float rval = route_key_value(rkey);
  const float lmax = __shfl_sync(0xffffffffu, rval, 0);
  const float z = (lane < k) ? expf(rval - lmax) : 0.0f;
  float sum = z;
#pragma unroll
  for (int off = 16; off > 0; off >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, off);
  *my_id = rid;
  *my_gate = z / sum;
}

// A lane's part of one k-block of one row group (half i of a unit, 16 rows x 64 K) from a ring slot, which holds the
// unit's codes and scales in the order of the tile (common.cuh): its operand pairs r0 (row R0) and r1 (row R1), 16
// values of K each. NF3 comes raw, with the two rows' scales as bf16 in the result; the others have their scales
// applied.
template <int FMT, int ACT>
__device__ __forceinline__ uint32_t decode_kblock(const uint8_t* slot, int i, int lane, uint32_t* r0, uint32_t* r1,
                                                  const uint32_t* s_scale, uint32_t nf3_lut) {
  if constexpr (FMT == FMT_NF3) {
    const uint32_t* v = reinterpret_cast<const uint32_t*>(slot) + 32 * i + lane;
    uint32_t s[4];
    nf3_selectors(v[0], v[64], v[128], s);
    nf3x8_lut(v[0], nf3_lut, r0);
    nf3x8_lut(v[64], nf3_lut, r0 + 4);
    nf3x8_lut(v[128], nf3_lut, r1);
    if constexpr (ACT == ACT_F16) nf3x8_to_f16x2(s[3], r1 + 4);
    else nf3x8_to_bf16x2(s[3], r1 + 4);
    return reinterpret_cast<const uint32_t*>(slot)[192 + 8 * i + (lane >> 2)];
  } else {
    const uint4 v = reinterpret_cast<const uint4*>(slot)[32 * i + lane];
    const uint32_t vv[4] = {v.x, v.y, v.z, v.w};
    uint32_t s0, s1;
    if constexpr (FMT == FMT_NVFP4) {
      const uint32_t sc = reinterpret_cast<const uint16_t*>(slot + 1024)[32 * i + lane];
      s0 = s_scale[sc & 0xFFu];
      s1 = s_scale[sc >> 8];
    } else {
      const uint32_t sc = reinterpret_cast<const uint16_t*>(slot + 1024)[16 * i + (lane >> 1)];
      s0 = s_scale[sc & 0xFFu];
      s1 = s_scale[sc >> 8];
    }
#pragma unroll
    for (int w = 0; w < 4; ++w) {
      uint32_t* p = (w < 2 ? r0 : r1) + 4 * (w & 1);
      if constexpr (ACT == ACT_F16) e2m1x8_to_f16x2(vv[w], p);
      else if constexpr (FMT == FMT_NVFP4) e2m1s_to_bf16x2(vv[w], p);
      else e2m1x8_to_bf16x2(vv[w], p);
    }
#pragma unroll
    for (int w = 0; w < 8; ++w) {
      r0[w] = mul_x2<ACT>(r0[w], s0);
      r1[w] = mul_x2<ACT>(r1[w], s1);
    }
    return 0;
  }
}

// One k-block's MMAs into the sums of one group of 8 columns.
template <int FMT, int ACT>
__device__ __forceinline__ void mma_kblock(const uint32_t* r0, const uint32_t* r1, uint32_t scales, const uint4& xa,
                                           const uint4& xb, float* acc) {
  const uint32_t xr[8] = {xa.x, xa.y, xa.z, xa.w, xb.x, xb.y, xb.z, xb.w};
  if constexpr (FMT == FMT_NF3) {
    float d[4];
    mma_16816_zc<ACT>(d, r0[0], r1[0], r0[1], r1[1], xr[0], xr[1]);
#pragma unroll
    for (int s = 1; s < 4; ++s)
      mma_16816<ACT>(d, r0[2 * s], r1[2 * s], r0[2 * s + 1], r1[2 * s + 1], xr[2 * s], xr[2 * s + 1]);
    const float s0 = __uint_as_float(scales << 16), s1 = __uint_as_float(scales & 0xFFFF0000u);
    acc[0] = fmaf(s0, d[0], acc[0]);
    acc[1] = fmaf(s0, d[1], acc[1]);
    acc[2] = fmaf(s1, d[2], acc[2]);
    acc[3] = fmaf(s1, d[3], acc[3]);
  } else {
#pragma unroll
    for (int s = 0; s < 4; ++s)
      mma_16816<ACT>(acc, r0[2 * s], r1[2 * s], r0[2 * s + 1], r1[2 * s + 1], xr[2 * s], xr[2 * s + 1]);
  }
}

// A lane's 16 bytes of the activations: only the lanes whose column exists load (a quarter of the warp, two columns,
// is one pass of shared memory); what the others hold is a column that nobody reads.
__device__ __forceinline__ void load_x(bool on, uint32_t x, int half, uint4& xa, uint4& xb) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %10, 0;\n\t"
      "@p ld.shared.v4.b32 {%0, %1, %2, %3}, [%8];\n\t"
      "@p ld.shared.v4.b32 {%4, %5, %6, %7}, [%9];\n\t}"
      : "+r"(xa.x), "+r"(xa.y), "+r"(xa.z), "+r"(xa.w), "+r"(xb.x), "+r"(xb.y), "+r"(xb.z), "+r"(xb.w)
      : "r"(x), "r"(x + half), "r"(on ? 1u : 0u)
      : "memory");
}

// A share's part of one group.
struct Segment {
  int g, loc, n, p0;  // its expert's place, slots and first position
  int a, b;           // units
  int act;            // byte offset of its activations
};

// Shared memory of decode_kernel.
template <int WARPS>
struct DkShared {
  uint8_t ring[WARPS][dk_ring(WARPS) * DK_SLOT];  // codes in flight; after a warp's last k-block its partial sums
  float part[WARPS][16][32];               // partial sums of the unit that a warp ended and another began
  uint32_t scale[256];                        // scale byte of the kept format -> pair of the operand type
  uint32_t nf3[DK_NF3_ENTRIES * 32];
  alignas(16) int id[DK_MAX_SLOTS];  // chosen experts by slot, then INT_MAX
  float gate[DK_MAX_SLOTS];
  int sorted[DK_MAX_SLOTS];    // slots by (expert, slot)
  int first[DK_MAX_SLOTS + 1]; // groups: first position in sorted
  int loc[DK_MAX_SLOTS];       // groups: their expert's entries of the layer's table
  float g13[DK_MAX_SLOTS], g2[DK_MAX_SLOTS];
  int cum[DK_MAX_SLOTS + 1];   // summed unit_cost of the groups before
  float hscale[DK_MAX_SLOTS];  // fp16: the power of two that a slot's h was divided by
  uint8_t head[DK_MAX_SLOTS];  // by position: a group begins
  uint32_t heads[DK_MAX_SLOTS / 32];
  int2 share[2][DK_MAX_SHARES + 1];  // of each product: where a share begins, a group and its unit
  int2 border[WARPS + 1];      // where a warp's part of the groups worked on begins: a group and its step
  int claim[2];                // the share worked on and the next one
  int abort, last;
};

constexpr int DK_SHARED_BYTES = (int)((sizeof(DkShared<DK_WARPS>) + 127) / 128 * 128);

__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_async_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

// Where a warp's copies into its ring stand: a step is STEP k-blocks of the segment's units, in their order.
struct Loader {
  const uint8_t* at;       // this lane's pieces of the next step
  const uint8_t* at2;
  uint32_t ring;           // shared address of the ring, at this lane's 16 bytes
  uint32_t slot;           // byte offset in it of the next step
  int u, in_unit, steps;   // unit, steps left of it and in all
};

// A lane's place in unit u, k-block kb. A unit's k-block is four runs of a tile in NF3 (3 x 256 bytes of codes, 64 of
// scales: 52 pieces of 16 bytes, a lane's at `at` and `at2`) and two in the kept formats (1024 bytes of codes, 128 or
// 64 of scales: a lane's two pieces at `at`, its third at `at2`).
template <int FMT>
__device__ __forceinline__ void loader_unit(Loader& l, const uint8_t* matrix, int KB, int kb, int lane) {
  const uint8_t* tile = matrix + ((size_t)(l.u >> 2) * KB + kb) * tile_bytes(FMT);
  const int i = l.u & 3;
  if constexpr (FMT == FMT_NF3) {
    l.at = tile + i * 256 + (lane >> 4) * 1024 + (lane & 15) * 16;
    l.at2 = tile + (lane < 16 ? 2 * 1024 + i * 256 + lane * 16 : 3 * 1024 + i * 64 + (lane & 3) * 16);
  } else {
    l.at = tile + i * 1024 + lane * 16;
    l.at2 = tile + 4096 + i * (FMT == FMT_NVFP4 ? 128 : 64) + (lane & 7) * 16;
  }
}

// Starts the next step's copies, if there is one; one commit group either way.
template <int FMT, int STEP, int RING>
__device__ __forceinline__ void loader_issue(Loader& l, int KB, int lane) {
  constexpr int TB = tile_bytes(FMT);
  if (l.steps > 0) {
    --l.steps;
    const uint32_t dst = l.ring + l.slot;
#pragma unroll
    for (int j = 0; j < STEP; ++j) {
      cp_async16(dst + j * DK_SLOT, l.at + j * TB);
      if (FMT != FMT_NF3) cp_async16(dst + j * DK_SLOT + 512, l.at + j * TB + 512);
    }
    if (lane < (FMT == FMT_NF3 ? 20 : (FMT == FMT_NVFP4 ? 8 : 4))) {
#pragma unroll
      for (int j = 0; j < STEP; ++j) cp_async16(dst + j * DK_SLOT + (FMT == FMT_NF3 ? 512 : 1024), l.at2 + j * TB);
    }
    l.slot = l.slot == (RING - STEP) * DK_SLOT ? 0 : l.slot + STEP * DK_SLOT;
    l.at += STEP * TB;
    l.at2 += STEP * TB;
    if (--l.in_unit == 0) {
      // the next quarter of the same tiles, or the first of those that follow
      const bool same = (++l.u & 3) != 0;
      const int codes = FMT == FMT_NF3 ? 256 : 1024, rest = FMT == FMT_NF3 ? (lane < 16 ? 256 : 64) : (FMT == FMT_NVFP4 ? 128 : 64);
      l.at += same ? codes - KB * TB : -3 * codes;
      l.at2 += same ? rest - KB * TB : -3 * rest;
      l.in_unit = KB / STEP;
    }
  }
  cp_async_commit();
}

template <int ACT, int KEPT, int WARPS>
struct DkCtx {
  const DecodeParams& p;
  DkShared<WARPS>& s;
  uint8_t* act;
  static constexpr int RING = dk_ring(WARPS);
  int ph, upg, KB, S, spu, cols_per_slot;  // S: k-blocks of a step; spu: steps of a unit
  int2 lo, hi;                             // the share: from a group's unit to another's

  __device__ __forceinline__ void set(int phase) {
    ph = phase;
    upg = (ph == 0 ? 2 * p.I : p.H) / DK_UNIT;
    KB = (ph == 0 ? p.H : p.I) / TILE_K;
    S = KB % 2 == 0 ? 2 : 1;
    spu = KB / S;
    cols_per_slot = ph == 0 ? 1 : 2;
  }

  __device__ __forceinline__ int fmt_of(int g) const { return (s.loc[g] & LOC_NF3) ? FMT_NF3 : KEPT; }

  // The part [lo, hi) of group g, of groups [g0, ...) worked on at once.
  __device__ __forceinline__ Segment segment(int g, int g0) const {
    Segment r;
    r.g = g;
    r.loc = s.loc[g];
    r.p0 = s.first[g];
    r.n = s.first[g + 1] - r.p0;
    r.a = g == lo.x ? lo.y : 0;
    r.b = g == hi.x ? hi.y : upg;
    r.act = (r.p0 - s.first[g0]) * slot_bytes();
    return r;
  }
  __device__ __forceinline__ int slot_bytes() const { return cols_per_slot * KB * 128; }  // of a slot's activations

  // Where share i begins: a group and its unit, the first whose cost begins at the share's or later.
  __device__ __forceinline__ int2 share_border(int i, int G) const {
    const int total = s.cum[G] * upg, each = div_by(total, p.by_shares);
    const int at = each * i + div_by((total - each * p.shares) * i, p.by_shares);  // total * i / shares
    int g = 0;
    for (int n = G; n > 0;) {  // the groups that end at `at` or before
      const int m = n >> 1;
      const bool ends = s.cum[g + m + 1] * upg <= at;
      g = ends ? g + m + 1 : g;
      n = ends ? n - m - 1 : m;
    }
    if (g == G) return make_int2(G, 0);
    const int fmt = fmt_of(g), u = by_unit_cost<KEPT, ACT>(at - s.cum[g] * upg + unit_cost<KEPT, ACT>(fmt) - 1, fmt);
    return u == upg ? make_int2(g + 1, 0) : make_int2(g, u);
  }
  // The group behind those that are worked on at once from g0 on: as many of the share as their activations fit, nearly
  // always all.
  __device__ __forceinline__ int end_of(int g0, int end) const {
    int g1 = g0 + 1;
    while (g1 < end && (s.first[g1 + 1] - s.first[g0]) * slot_bytes() <= p.act_cap) ++g1;
    return g1;
  }
  // Where warp w's part of the groups [g0, g1) begins, an even part of their cost: a group and its step.
  __device__ __forceinline__ int2 part_border(int w, int g0, int g1) const {
    const int base = s.cum[g0];
    auto cost = [&](int g, int u) { return ((s.cum[g] - base) * upg + (u ? u * (s.cum[g + 1] - s.cum[g]) : 0)) * spu; };
    const int from = g0 == lo.x ? cost(g0, lo.y) : 0, to = g1 > hi.x ? cost(hi.x, hi.y) : cost(g1, 0);
    const int at = from + (int)((long long)(to - from) * w / WARPS);
    int g = g0;
    while (g + 1 < g1 && cost(g + 1, 0) <= at) ++g;
    return make_int2(g, by_unit_cost<KEPT, ACT>(at - cost(g, 0), fmt_of(g)) - (g == lo.x ? lo.y * spu : 0));
  }

  // Activations of one segment as MMA fragments: [k-block][half][column][q], 16 bytes each: k = 16 q + 8 half + 0..7.
  __device__ __forceinline__ void fill(const Segment& r) const {
    const int tid = threadIdx.x;
    uint8_t* dst = act + r.act;
    if (ph == 0) {
      const int pieces = p.H / 8;
      for (int c = 0; c < r.n; ++c) {
        const uint4* src = reinterpret_cast<const uint4*>(p.x + (size_t)(s.sorted[r.p0 + c] / p.topk) * p.H);
        for (int i = tid; i < pieces; i += WARPS * 32)
          *reinterpret_cast<uint4*>(dst + (((i >> 3) * 2 + (i & 1)) * r.n + c) * 64 + ((i >> 1) & 3) * 16) = __ldca(src + i);
      }
    } else {
      const int pieces = p.I / 8, cols = 2 * r.n;
      for (int c = 0; c < r.n; ++c) {
        const int slot = s.sorted[r.p0 + c];
        const float4* src = reinterpret_cast<const float4*>(p.h + (size_t)slot * p.I);
        float down = 1.0f;
        if constexpr (ACT == ACT_F16) {
          // the power of two that brings the largest |h| to 2^14 .. 2^15; what is not finite has none
          const uint32_t m = __ldcg(p.hmax + slot);
          const int ex = (int)(m >> 23);
          const int by = ex == 0 || ex >= 255 ? 0 : min(126, max(-126, 14 + 127 - ex));
          down = __uint_as_float((uint32_t)(127 + by) << 23);
          if (tid == 0) s.hscale[r.p0 + c] = __uint_as_float((uint32_t)(127 - by) << 23);
        }
        for (int i = tid; i < pieces; i += WARPS * 32) {
          const float4 v0 = __ldcg(src + 2 * i), v1 = __ldcg(src + 2 * i + 1);
          const float v[8] = {v0.x, v0.y, v0.z, v0.w, v1.x, v1.y, v1.z, v1.w};
          uint32_t hi4[4], lo4[4];
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const float a = v[2 * j] * down, b = v[2 * j + 1] * down;
            hi4[j] = f32_to_act_x2<ACT>(a, b);
            const float2 back = act_x2_to_f32<ACT>(hi4[j]);
            // an infinite hi has no rest
            lo4[j] = f32_to_act_x2<ACT>(isinf(back.x) ? 0.0f : a - back.x, isinf(back.y) ? 0.0f : b - back.y);
          }
          uint8_t* at = dst + (((i >> 3) * 2 + (i & 1)) * cols + 2 * c) * 64 + ((i >> 1) & 3) * 16;
          *reinterpret_cast<uint4*>(at) = make_uint4(hi4[0], hi4[1], hi4[2], hi4[3]);
          *reinterpret_cast<uint4*>(at + 64) = make_uint4(lo4[0], lo4[1], lo4[2], lo4[3]);
        }
      }
    }
  }

  // Results of row group u: rows R0 = 16 u + g and R1 = R0 + 8 (tile order).
  __device__ __forceinline__ void emit(const Segment& r, int u, float (*acc)[4]) const {
    const float gsc = (ph == 0 ? s.g13[r.g] : s.g2[r.g]) * (KEPT == FMT_NVFP4 && !(r.loc & LOC_NF3) ? nvfp4_unscale<ACT>() : 1.0f);
    const int lane = threadIdx.x & 31, g = lane >> 2, q = lane & 3;
    if (ph == 0) {
      const int ch = u * 8 + g;
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        const int col = 2 * q + c;
        const float z = acc[0][c] * gsc, v = silu_f(z) * (acc[0][2 + c] * gsc);
        const bool there = col < r.n;
        const int slot = there ? s.sorted[r.p0 + col] : 0;
        if (there) p.h[(size_t)slot * p.I + ch] = v;
        if constexpr (ACT == ACT_F16) {
          uint32_t m = there ? __float_as_uint(v) & 0x7FFFFFFFu : 0u;
#pragma unroll
          for (int off = 4; off < 32; off <<= 1) m = max(m, __shfl_xor_sync(0xffffffffu, m, off));
          if (there && g == 0) atomicMax(p.hmax + slot, m);
        }
      }
    } else {
#pragma unroll
      for (int n = 0; n < 2; ++n) {
        const int c = 4 * n + q;
        if (c >= r.n) continue;
        const float by = ACT == ACT_F16 ? gsc * s.hscale[r.p0 + c] : gsc;
        float* y = p.y + (size_t)s.sorted[r.p0 + c] * p.H + 16 * u + g;
        y[0] = (acc[n][0] + acc[n][1]) * by;
        y[8] = (acc[n][2] + acc[n][3]) * by;
      }
    }
  }

  __device__ __forceinline__ int spu_of(int steps) const { return div_by(steps, ph == 0 ? p.by_spu13 : p.by_spu2); }

  // The first copies of this warp's steps [from, to) of a segment.
  template <int FMT, int STEP>
  __device__ __forceinline__ void begin(Loader& l, const Segment& r, int from, int to, int warp, int lane) const {
    constexpr bool nf3 = FMT == FMT_NF3;
    const uint8_t* matrix = (nf3 ? p.nf3_buf : p.kept_buf) +
            (size_t)(r.loc & 0x7FFF) * (nf3 ? p.nf3_expert_bytes : p.kept_expert_bytes) +
            (ph == 0 ? 0 : (nf3 ? p.nf3_w2_off : p.kept_w2_off));
    l.ring = smem_u32(s.ring[warp]) + lane * 16;
    l.slot = 0;
    const int whole = spu_of(from), rest = from - whole * spu;
    l.u = r.a + whole;
    l.in_unit = spu - rest;
    l.steps = to - from;
    loader_unit<FMT>(l, matrix, KB, rest * STEP, lane);
#pragma unroll 1
    for (int i = 0; i < RING / STEP - 1; ++i) loader_issue<FMT, STEP, RING>(l, KB, lane);
  }

  // This warp's steps [from, to) of a segment, whose first copies are under way. Whole units are emitted; the sums of
  // one that another warp began go to s.part, of one that another ends to the ring.
  template <int FMT, int STEP, bool TWO>
  __device__ __forceinline__ void run(Loader& l, const Segment& r, int from, int to, int warp, int lane) const {
    constexpr int SLOTS = RING / STEP;
    const int g = lane >> 2, q = lane & 3;
    const uint32_t nf3_lut = smem_u32(s.nf3) + 4u * (uint32_t)lane;
    const int cols = r.n * cols_per_slot, half = cols * 64;
    const bool on = g < cols, on2 = g + 8 < cols;
    const uint32_t x0 = smem_u32(act) + r.act + g * 64 + q * 16;
    const uint32_t* const s_scale = s.scale;
    const uint8_t* const ring = s.ring[warp];
    const uint8_t* w = ring;
    int u = spu_of(from), st = from - u * spu;
    u += r.a;
    bool whole = st == 0;
    uint32_t x = x0 + st * STEP * 2 * half;
    uint4 xa = make_uint4(0, 0, 0, 0), xb = xa;
    float acc[2][2][4] = {};  // of each row group, of each group of 8 columns
    for (int left = to - from; left > 0; --left) {
      cp_async_wait<SLOTS - 2>();
      __syncwarp();
      loader_issue<FMT, STEP, RING>(l, KB, lane);  // into the slot of the step before, which every lane has read
#pragma unroll
      for (int j = 0; j < STEP; ++j) {
        uint32_t r0[2][8], r1[2][8], sc[2];
#pragma unroll
        for (int i = 0; i < 2; ++i)
          sc[i] = decode_kblock<FMT, ACT>(w + j * DK_SLOT, i, lane, r0[i], r1[i], s_scale, nf3_lut);
        load_x(on, x, half, xa, xb);
#pragma unroll
        for (int i = 0; i < 2; ++i) mma_kblock<FMT, ACT>(r0[i], r1[i], sc[i], xa, xb, acc[i][0]);
        if constexpr (TWO) {  // more than 8 columns
          load_x(on2, x + 512, half, xa, xb);
#pragma unroll
          for (int i = 0; i < 2; ++i) mma_kblock<FMT, ACT>(r0[i], r1[i], sc[i], xa, xb, acc[i][1]);
        }
        x += 2 * half;
      }
      w = w == ring + (RING - STEP) * DK_SLOT ? ring : w + STEP * DK_SLOT;
      if (++st == spu) {
        if (whole) {
#pragma unroll
          for (int i = 0; i < 2; ++i) emit(r, 2 * u + i, acc[i]);
        } else {
          put(s.part[warp][0], lane, acc);
        }
        whole = true;
        st = 0;
        ++u;
        x = x0;
#pragma unroll
        for (int i = 0; i < 16; ++i) acc[i >> 3][(i >> 2) & 1][i & 3] = 0.0f;
      }
    }
    __syncwarp();
    if (st != 0) put(reinterpret_cast<float*>(s.ring[warp]), lane, acc);
  }
  static __device__ __forceinline__ void put(float* at, int lane, float (*acc)[2][4]) {
#pragma unroll
    for (int i = 0; i < 16; ++i) at[i * 32 + lane] = acc[i >> 3][(i >> 2) & 1][i & 3];
  }

  // The unit that this warp ended and others began: their sums in the order of K.
  __device__ __forceinline__ void join(int2 from, int2 to, int g0, int g1, int warp, int lane) const {
    const int u = spu_of(from.y), begin = u * spu;
    if (from.x >= g1 || from.y == begin || (to.x == from.x && to.y < begin + spu)) return;
    const Segment r = segment(from.x, g0);
    int v = warp - 1;  // the warp that began it
    while (s.border[v].x == from.x && s.border[v].y > begin) --v;
    float acc[2][2][4] = {};
    auto add = [&](const float* sums) {
#pragma unroll
      for (int i = 0; i < 16; ++i) acc[i >> 3][(i >> 2) & 1][i & 3] += sums[i * 32 + lane];
    };
    for (; v < warp; ++v) {
      const int2 at = s.border[v], end = s.border[v + 1];
      if (at.x == end.x && at.y == end.y) continue;  // a warp without work
      add(reinterpret_cast<const float*>(s.ring[v]));
    }
    add(s.part[warp][0]);
#pragma unroll
    for (int i = 0; i < 2; ++i) emit(r, 2 * (r.a + u) + i, acc[i]);
  }
};

template <int ACT, int KEPT, int WARPS>
__global__ void __launch_bounds__(WARPS * 32, 1) decode_kernel(const __grid_constant__ DecodeParams p) {
  extern __shared__ __align__(128) uint8_t smem[];
  constexpr int THREADS = WARPS * 32;
  static_assert(THREADS >= DK_MAX_SLOTS && WARPS >= DECODE_MAX_TOKENS && WARPS < 32, "a thread a slot, a warp a token");
  static_assert(sizeof(DkShared<WARPS>) <= DK_SHARED_BYTES, "what the activations leave");
  DkShared<WARPS>& s = *reinterpret_cast<DkShared<WARPS>*>(smem);
  uint8_t* act = smem + DK_SHARED_BYTES;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int S = p.T * p.topk;
  if (tid < 256)
    s.scale[tid] = KEPT == FMT_NVFP4 ? e4m3_lut_entry<ACT>((uint32_t)tid)
                                     : bf16_bcast(ACT == ACT_F16 ? e8m0_to_f16((uint32_t)tid) : e8m0_to_bf16((uint32_t)tid));
  if (p.has_nf3)
    for (int w = tid; w < DK_NF3_ENTRIES * 32; w += THREADS) {
      uint32_t v[4];
      if constexpr (ACT == ACT_F16) nf3x8_to_f16x2((uint32_t)(w >> 5) & 0x77u, v);
      else nf3x8_to_bf16x2((uint32_t)(w >> 5) & 0x77u, v);
      s.nf3[w] = v[0];
    }
  if (tid < DK_MAX_SLOTS) {
    s.id[tid] = INT_MAX;
    s.head[tid] = 0;
  }
  if (tid == 0) s.abort = 0;
  // The layer's table while the router still runs: constants at an index of each thread's own are read one by one.
  ExpertTable& tab = *reinterpret_cast<ExpertTable*>(s.ring);  // which the weights take later
  static_assert(sizeof(ExpertTable) <= sizeof(s.ring), "the table in the rings");
  for (int e = tid; e < p.E; e += THREADS) {
    tab.loc[e] = p.tab.loc[e];
    tab.g13[e] = p.tab.g13[e];
    tab.g2[e] = p.tab.g2[e];
  }
  __syncthreads();
  pdl_wait();  // the router's logits; also the last use of the workspace
  pdl_trigger();
  if (tid == THREADS - 1) s.claim[0] = atomicAdd(p.ctl, 1);
  if (warp < p.T) {
    int id;
    float gt;
    warp_route_few(p.logits + (size_t)warp * p.E, p.E, p.topk, lane, &id, &gt);
    if (lane < p.topk) {
      const int slot = warp * p.topk + lane;
      s.id[slot] = id;
      s.gate[slot] = gt;
      if (blockIdx.x == 0) {
        if (p.ids) p.ids[slot] = id;
        if (p.gates) p.gates[slot] = gt;
      }
    }
  }
  __syncthreads();
  // Slots by (expert, slot), and groups of up to group_tokens slots of one expert (an expert has at most T).
  if (tid < S) {
    const int e = s.id[tid];
    int less = 0, same = 0;
    for (int o = 0; o < S; o += 4) {
      const int4 f = *reinterpret_cast<const int4*>(s.id + o);
      less += (f.x < e) + (f.y < e) + (f.z < e) + (f.w < e);
      same += (f.x == e && o < tid) + (f.y == e && o + 1 < tid) + (f.z == e && o + 2 < tid) + (f.w == e && o + 3 < tid);
    }
    s.sorted[less + same] = tid;
    if (same % p.group_tokens == 0) s.head[less + same] = 1;
  }
  __syncthreads();
  const uint32_t ballot = __ballot_sync(0xffffffffu, tid < S && s.head[tid]);
  if (lane == 0 && warp < DK_MAX_SLOTS / 32) s.heads[warp] = ballot;
  __syncthreads();
  int G = 0;
  {
    int before = 0;
#pragma unroll
    for (int w = 0; w < DK_MAX_SLOTS / 32; ++w) {
      const int h = __popc(s.heads[w]);
      if (w < warp) before += h;
      G += h;
    }
    if (tid < S && s.head[tid]) {
      const int g = before + __popc(ballot & ((1u << lane) - 1u));
      const int e = s.id[s.sorted[tid]];
      s.first[g] = tid;
      s.loc[g] = tab.loc[e];
      s.g13[g] = tab.g13[e];
      s.g2[g] = tab.g2[e];
    }
    if (tid == 0) s.first[G] = S;
  }
  __syncthreads();
  if (warp == 0) {
    int run = 0;
    for (int g0 = 0; g0 < G; g0 += 32) {
      const int g = g0 + lane;
      const int w = g < G ? unit_cost<KEPT, ACT>((s.loc[g] & LOC_NF3) ? FMT_NF3 : KEPT) : 0;
      int incl = w;
#pragma unroll
      for (int off = 1; off < 32; off <<= 1) {
        const int nb = __shfl_up_sync(0xffffffffu, incl, off);
        if (lane >= off) incl += nb;
      }
      if (g < G) s.cum[g] = run + incl - w;
      run += __shfl_sync(0xffffffffu, incl, 31);
    }
    if (lane == 0) s.cum[G] = run;
  }
  __syncthreads();

  const int C = p.shares;
  int* done13 = p.ctl + DK_CTL_DONE;
  int* done2 = p.ctl + DK_CTL_DONE2;
  const int upg13 = 2 * p.I / DK_UNIT;
  for (int i = tid; i <= 2 * C + 1; i += THREADS) {
    DkCtx<ACT, KEPT, WARPS> c{p, s, act};
    const int ph = i > C ? 1 : 0;
    c.set(ph);
    s.share[ph][i - ph * (C + 1)] = c.share_border(i - ph * (C + 1), G);
  }
  __syncthreads();
  for (int place = 0;; place ^= 1) {
    const int claim = s.claim[place];
    if ((unsigned)claim >= 2u * (unsigned)C) break;  // all taken (or a workspace that was not zeroed)
    DkCtx<ACT, KEPT, WARPS> c{p, s, act};
    c.set(claim >= C ? 1 : 0);
    c.lo = s.share[c.ph][claim - c.ph * C];
    c.hi = s.share[c.ph][claim - c.ph * C + 1];
    int g0 = c.lo.x;
    const int gend = c.lo.x == c.hi.x && c.lo.y == c.hi.y ? g0 : (c.hi.y > 0 ? c.hi.x + 1 : c.hi.x);
    if (g0 == gend) {  // a share without units
      if (tid == THREADS - 1) s.claim[place ^ 1] = atomicAdd(p.ctl, 1);
      __syncthreads();
    }
    while (g0 < gend) {
      const int g1 = c.end_of(g0, gend);
      const int2 mine = c.part_border(warp + (lane & 1), g0, g1);
      if (lane < 2) s.border[warp + lane] = mine;  // for join (the next warp writes the same)
      const int2 from = make_int2(__shfl_sync(0xffffffffu, mine.x, 0), __shfl_sync(0xffffffffu, mine.y, 0));
      const int2 to = make_int2(__shfl_sync(0xffffffffu, mine.x, 1), __shfl_sync(0xffffffffu, mine.y, 1));
      Loader l;
      auto range = [&](int g) {
        const int all = g >= g1 ? 0 : ((g == c.hi.x ? c.hi.y : c.upg) - (g == c.lo.x ? c.lo.y : 0)) * c.spu;
        return make_int2(g == from.x ? from.y : 0, g == to.x ? to.y : all);
      };
      // f(format, k-blocks of a step) of a segment, as types
      auto as = [&](const Segment& r, auto f) {
        using std::integral_constant;
        auto by_step = [&](auto fmt) {
          if (c.S == 2) f(fmt, integral_constant<int, 2>());
          else f(fmt, integral_constant<int, 1>());
        };
        if (r.loc & LOC_NF3) by_step(integral_constant<int, FMT_NF3>());
        else by_step(integral_constant<int, KEPT>());
      };
      auto start = [&](const Segment& r, int2 steps) {
        as(r, [&](auto fmt, auto step) { c.template begin<fmt(), step()>(l, r, steps.x, steps.y, warp, lane); });
      };
      int i = from.x;
      while (i < to.x && range(i).x >= range(i).y) ++i;
      const int first = i;
      if (range(first).x < range(first).y) start(c.segment(first, g0), range(first));
      // the next share's way to L2 and back under this one's work
      if (g0 == c.lo.x && tid == THREADS - 1) s.claim[place ^ 1] = atomicAdd(p.ctl, 1);
      if (c.ph == 1) {
        // every W13 unit of these groups written, by any CTA
        if (warp == 0)
          for (int g = g0 + lane; g < g1; g += 32)
            if (!wait_count_at_least(done13 + g, upg13, &s.abort, p.wait_limit_ns)) {
              *(volatile int*)&s.abort = 1;
              set_status(p.status, DEV_TIMEOUT);
            }
        __syncthreads();
        if (*(volatile int*)&s.abort) {  // the caller reads the status
          cp_async_wait<0>();
          return;
        }
      }
      for (int g = g0; g < g1; ++g) c.fill(c.segment(g, g0));
      __syncthreads();
      for (; i <= to.x && i < g1; ++i) {
        const int2 r = range(i);
        if (r.x >= r.y) continue;
        const Segment g = c.segment(i, g0);
        if (i != first) start(g, r);
        as(g, [&](auto fmt, auto step) {
          if (g.n * c.cols_per_slot > 8) c.template run<fmt(), step(), true>(l, g, r.x, r.y, warp, lane);
          else c.template run<fmt(), step(), false>(l, g, r.x, r.y, warp, lane);
        });
      }
      __syncthreads();
      c.join(from, to, g0, g1, warp, lane);
      __threadfence();  // this thread's h or y values, before their counts
      __syncthreads();
      if (c.ph == 0) {
        for (int g = g0 + tid; g < g1; g += THREADS) {
          const Segment r = c.segment(g, g0);
          atomicAdd(done13 + g, r.b - r.a);
        }
      } else if (tid == 0) {
        int units = 0;
        for (int g = g0; g < g1; ++g) {
          const Segment r = c.segment(g, g0);
          units += r.b - r.a;
        }
        atomicAdd(done2, units);
      }
      g0 = g1;
    }
  }
  // Every share is taken, by CTAs that run: when their units are done, each CTA sums the slots of its part of the columns.
  if (tid == 0 && !wait_count_at_least(done2, G * (p.H / DK_UNIT), &s.abort, p.wait_limit_ns)) {
    *(volatile int*)&s.abort = 1;
    set_status(p.status, DEV_TIMEOUT);
  }
  __syncthreads();
  if (*(volatile int*)&s.abort) return;
  const int half = p.H / 2, pairs = p.T * half, each = (pairs + (int)gridDim.x - 1) / (int)gridDim.x;  // pairs of columns
  for (int j = (int)blockIdx.x * each + tid; j < min(pairs, ((int)blockIdx.x + 1) * each); j += THREADS) {
    const int t = j / half, col = 2 * (j - t * half);
    const float* y = p.y + (size_t)t * p.topk * p.H + col;
    float a = 0.0f, b = 0.0f;
#pragma unroll 8
    for (int k = 0; k < p.topk; ++k) {
      const float2 v = __ldcg(reinterpret_cast<const float2*>(y + (size_t)k * p.H));
      const float gt = s.gate[t * p.topk + k];
      a = fmaf(gt, v.x, a);
      b = fmaf(gt, v.y, b);
    }
    *reinterpret_cast<uint32_t*>(p.out + (size_t)t * p.H + col) = f32x2_to_act<ACT>(a, b);
  }
  // The last CTA to leave brings the workspace's counters back to zero.
  if (tid == 0) s.last = atomicAdd(p.ctl + 1, 1) == (int)gridDim.x - 1 ? 1 : 0;
  __syncthreads();
  if (s.last) {
    for (int i = tid; i < G; i += THREADS) done13[i] = 0;
    if (ACT == ACT_F16)
      for (int i = tid; i < S; i += THREADS) p.hmax[i] = 0;
    if (tid < 2) p.ctl[tid] = 0;
    if (tid == 2) *done2 = 0;
  }
}

// ------------------------------------------------------------ launch
int decode_act_cap() { return DK_SMEM_LIMIT - DK_SHARED_BYTES; }

template <int ACT, int TM>
static cudaError_t launch_router(const DecodeParams& p, const uint16_t* router, const float* bias, cudaStream_t st) {
  return launch_pdl(router_kernel<ACT, TM>, dim3(p.E), dim3(RK_THREADS), 0, st, p.x, router, bias, p.T, p.H, p.E,
                    p.logits);
}

template <int ACT, int KEPT, int WARPS>
static cudaError_t launch_decode_warps(const DecodeParams& p, int num_sms, cudaStream_t st) {
  static std::atomic<unsigned long long> attr{0};
  cudaError_t e = ensure_smem_attr(decode_kernel<ACT, KEPT, WARPS>, DK_SMEM_LIMIT, attr);
  if (e == cudaSuccess) e = launch_pdl(decode_kernel<ACT, KEPT, WARPS>, dim3(num_sms), dim3(WARPS * 32), DK_SMEM_LIMIT, st, p);
  return e;
}

template <int ACT, int KEPT>
static cudaError_t launch_decode_as(const DecodeParams& p, const uint16_t* router, const float* bias, int num_sms,
                                     cudaStream_t st) {
  cudaError_t e =
      p.T == 1 ? launch_router<ACT, 1>(p, router, bias, st)
                 : (p.T == 2 ? launch_router<ACT, 2>(p, router, bias, st)
                             : (p.T <= 4 ? launch_router<ACT, 4>(p, router, bias, st) : launch_router<ACT, 8>(p, router, bias, st)));
  if (e != cudaSuccess) return e;
  const long long steps = (long long)p.T * p.topk * (2 * p.I / DK_UNIT) * (p.H / (2 * TILE_K));  // of W13, at most
  e = steps <= (long long)DK_FEW_STEPS * num_sms ? launch_decode_warps<ACT, KEPT, DK_FEW_WARPS>(p, num_sms, st)
                                                 : launch_decode_warps<ACT, KEPT, DK_WARPS>(p, num_sms, st);
  count_launches(2);
  return e;
}

cudaError_t launch_decode(const DecodeParams& p, const uint16_t* router, const float* bias, int num_sms, cudaStream_t st) {
  auto launch = p.act_type == ACT_F16
                    ? (p.kept_fmt == FMT_NVFP4 ? launch_decode_as<ACT_F16, FMT_NVFP4> : launch_decode_as<ACT_F16, FMT_MXFP4>)
                    : (p.kept_fmt == FMT_NVFP4 ? launch_decode_as<ACT_BF16, FMT_NVFP4> : launch_decode_as<ACT_BF16, FMT_MXFP4>);
  return launch(p, router, bias, num_sms, st);
}

}  // namespace hmoe
