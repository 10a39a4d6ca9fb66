// lora.cu -- low-rank adapters of many requests beside a shared projection:
//   out[t] = base[t] + scale_a * B_a (A_a x[t]),  a = ids[t] (-1: none).
//
// What a batch cannot do without: x, base and each used adapter read once, out
// written once. That bounds every size: at rank 128 the products are 128
// operations for a byte of x, base or out (B u's two parts counted), of which
// the tensor cores do about 290 in a byte's time at HBM.
//
// u = A x is summed in fp32 and enters the second product as the sum of two
// values of the activation type (split_act): u then keeps 16 bits in bf16, 22 in
// fp16 (ROW_POWERS), and out has one rounding, its own. One 16-bit u would add an
// error as large as that. No sum's order depends on the schedule.
//
// Two ways, by what the host knows of the batch (lora_planned_small): a kernel
// that serves 16 rows of one adapter with a small cluster, whose time is
// latency (one launch up to 2048 rows, two above), and a pair of persistent
// tensor-core kernels over tiles of 128 rows of one adapter (three launches).
#include <math.h>

#include "act.cuh"
#include "common.cuh"
#include "internal.h"
#include "tcgen05.cuh"

namespace hmoe {

// ------------------------------------------------------------ the packed adapters
// Byte of A[r][k] in the block of an adapter of rank r16 (128-byte swizzle:
// the 16-byte chunks of row r are permuted by r % 8).
__host__ __device__ __forceinline__ size_t lora_a_byte(int r16, int r, int k) {
  const int chunk = ((k >> 3) & 7) ^ (r & 7);
  return ((size_t)(k >> 6) * r16 + r) * 128 + chunk * 16 + (k & 7) * 2;
}
// Byte of B[n][r] from the start of the block's B tiles. The rows of a tile are
// permuted inside each 32: row 8 q + 2 j + e lies at 8 j + 2 q + e. Where an
// accumulator gives a lane the columns 8 j + 2 q + e of q fixed, as mma.sync and
// the 16x256b loads from tensor memory do, these are 8 neighbouring columns of
// the result: 16 bytes of a row, loaded and stored without shared memory.
__host__ __device__ __forceinline__ size_t lora_b_byte(int r16, int n, int r) {
  const int at = (n & 32) + ((n >> 1) & 3) * 8 + ((n >> 3) & 3) * 2 + (n & 1);
  return (size_t)(n >> 6) * r16 * 128 + ((size_t)(r >> 3) * 64 + at) * 16 + (r & 7) * 2;
}

__global__ void lora_clear_kernel(uint32_t* words, int n) {
  pdl_wait();
  pdl_trigger();
  for (int i = blockIdx.x * blockDim.x + threadIdx.x; i < n; i += gridDim.x * blockDim.x) words[i] = 0u;
}

cudaError_t launch_lora_clear(const LoraGeom& g, uint8_t* packed, cudaStream_t st) {
  const int n = (int)(g.block_off / 4);
  cudaError_t e = launch_pdl(lora_clear_kernel, dim3(1), dim3(256), 0, st, reinterpret_cast<uint32_t*>(packed), n);
  count_launches(1);
  return e;
}

// One thread per 16-byte chunk of the slot's tiles: 8 values along K of A, or
// 8 along the rank of B; zeros past the rank, K and N.
__global__ void lora_load_kernel(LoraGeom g, uint8_t* packed, int slot, const uint16_t* __restrict__ A,
                                 const uint16_t* __restrict__ B, int rank, float scale) {
  pdl_wait();
  pdl_trigger();
  const int r16 = (rank + 15) / 16 * 16;
  uint8_t* block = packed + g.block_off + (size_t)slot * g.block_bytes;
  if (blockIdx.x == 0 && threadIdx.x == 0) {
    reinterpret_cast<int*>(packed)[slot] = rank;
    reinterpret_cast<float*>(packed + g.scale_off)[slot] = scale;
  }
  const long long na = (long long)g.KB * r16 * 8, nb = (long long)g.NB * r16 * 8;
  for (long long i = blockIdx.x * (long long)blockDim.x + threadIdx.x; i < na + nb;
       i += (long long)gridDim.x * blockDim.x) {
    uint16_t v[8];
    uint8_t* dst;
    if (i < na) {
      const int kb = (int)(i / (r16 * 8)), rem = (int)(i % (r16 * 8));
      const int r = rem >> 3, k0 = kb * 64 + (rem & 7) * 8;
#pragma unroll
      for (int j = 0; j < 8; ++j) v[j] = (r < rank && k0 + j < g.K) ? A[(size_t)r * g.K + k0 + j] : (uint16_t)0;
      dst = block + lora_a_byte(r16, r, k0);
    } else {
      const long long b = i - na;
      const int nt = (int)(b / (r16 * 8)), rem = (int)(b % (r16 * 8));
      const int n = nt * 64 + rem / (r16 / 8), r0 = (rem % (r16 / 8)) * 8;
#pragma unroll
      for (int j = 0; j < 8; ++j) v[j] = (n < g.N && r0 + j < rank) ? B[(size_t)n * rank + r0 + j] : (uint16_t)0;
      dst = block + g.b_off + lora_b_byte(r16, n, r0);
    }
    *reinterpret_cast<uint4*>(dst) = *reinterpret_cast<const uint4*>(v);
  }
}

cudaError_t launch_lora_load(const LoraGeom& g, uint8_t* packed, int slot, const uint16_t* A, const uint16_t* B,
                             int rank, float scale, cudaStream_t st) {
  const int r16 = (rank + 15) / 16 * 16;
  const long long chunks = (long long)(g.KB + g.NB) * r16 * 8;
  const long long blocks = (chunks + 255) / 256;
  const dim3 grid((unsigned)(blocks < 1 ? 1 : (blocks < 1024 ? blocks : 1024)));
  cudaError_t e = launch_pdl(lora_load_kernel, grid, dim3(256), 0, st, g, packed, slot, A, B, rank, scale);
  count_launches(1);
  return e;
}

// ------------------------------------------------------------ forward
template <int ACT>
__device__ __forceinline__ float act_f32(uint16_t b) {
  if constexpr (ACT == ACT_F16) return __half2float(__ushort_as_half(b));
  else return bf16_bits_to_float(b);
}

// The adapter of row t: its slot, or -1 where the row has none or an id out of
// range (which is recorded).
__device__ __forceinline__ int lora_slot(const LoraParams& p, int t) {
  const int a = p.ids[t];
  if (a >= p.g.slots || a < -1) {
    set_status(p.status, DEV_BAD_ROUTE);
    return -1;
  }
  return a;
}

// ------------------------------------------------------------ small batches: one launch
// A cluster of C CTAs serves up to LS_TOK rows of one adapter: CTA c sums A x
// over its share of K, the CTAs exchange their partial sums through
// distributed shared memory, and each adds B u for its share of N. The batch
// is grouped without a pass of its own: up to LS_MAX_T rows, cluster t belongs to
// row t, and goes on only if row t is the first of a group, that is if the number
// of earlier rows with the same id is a multiple of LS_TOK (256 rows of 8 adapters
// of rank 64, 6144x6144: 17.5 us, counted as below 15.8; 64 rows 14.6, counted
// 16.0).
//
// What the busiest SM fetches bounds it where the batch is large (64 rows of 64
// adapters of ranks 1 to 64, 6144x6144: 33 MB in 14.0 us, but two CTAs of rank 64
// on one SM fetch 512 KB, at 30 to 36 KB a us however many loads are in flight:
// rings of bulk copies took 16.7 us); below, a chain of waits does:
// ids, A and x, the cluster's exchange, B (one row of rank 16, 2048x2048: 3.9 us,
// of rank 64, 6144x6144, from L2: 8.0 us). So a CTA has the next step's operands on their
// way, B's first ones and the base's before the exchange, and only the group's
// own rows are exchanged. (Asking L2 for B at the start made 64 rows 2 us slower:
// it delays A.)
//
// Both products run on mma.sync m16n8k16, whose 16 rows suit a group (tcgen05's
// smallest M is 64, and would want the weights staged in shared memory first),
// with the rows on the M side and the weights, straight from global memory, on
// the N side. K inside a group of 32
// (and the rank in the second product) is permuted alike for both operands, so
// that a lane's operand words are 16 bytes of one row. The columns of the
// second product are permuted so that a lane ends up with 8 neighbouring ones
// (lora_b_byte).
constexpr int LS_THREADS = 256;
constexpr int LS_WARPS = LS_THREADS / 32;
constexpr int LS_TOK = 16;
constexpr int LS_MAX_T = LORA_ONE_LAUNCH_ROWS;
static_assert(LS_MAX_T <= LS_THREADS, "the grouping looks at one row a thread");
// CTAs of an SM, by the registers of the kernel for this rank.
constexpr int ls_per_sm(int r16) { return r16 <= 64 ? 2 : 1; }
// What a batch is likely to look like, from what the host knows of it: rows
// that draw their adapters at random from the slots have slots (1 - exp(-T /
// slots)) of them, and each makes about max(1, rows / 16 + 0.47) groups.
struct LoraBatch {
  double adapters, rows, groups;  // rows: of one adapter
};
inline LoraBatch lora_batch(const LoraGeom& g, int T) {
  LoraBatch b;
  b.adapters = g.slots * (1.0 - exp(-(double)T / g.slots));
  b.rows = T / b.adapters;
  b.groups = b.adapters * fmax(1.0, b.rows / LS_TOK + 0.47);
  return b;
}
// CTAs of a cluster, 2 to 8: as many as let the groups run in one wave, by how
// many clusters of a size run at once (fits[c]; a cluster stays in one part of
// the chip, so 43 of 7 do not run at once on 152 SMs with two CTAs each). A
// group of more CTAs is a shorter wait, a second wave is another: 64 rows of 64
// adapters of rank 64, 6144x6144 took 17.9, 14.6 and 17.3 us with 4, 6 and 8; 128
// of 128, rank 32, 16.9, 20.0 and 23.1 with 3, 4 and 8; 1024 of 64 38.1, 30.6 and
// 39.1 with 2, 3 and 4; 581 of 7, rank 13, 176x768, 7.9 and 12.7 with 6 and 7;
// one row 8.3, 6.7 and 6.1 with 4, 6 and 8.
// Where the adapters are small and each row has a cluster of its own, starting
// the clusters is what counts: 256 CTAs in all (64 rows of rank 16, 2048x2048:
// 4.9, 5.8 and 7.4 us with 4, 6 and 8).
constexpr int LS_MAX_CLUSTER = 8;
inline int ls_cluster(const LoraGeom& g, int T, const int* fits) {
  const double groups = lora_batch(g, T).groups;
  int c = LS_MAX_CLUSTER;
  while (c > 2 && fits[c] < 1.02 * groups) --c;
  if (T <= LS_MAX_T && (long long)(g.KB + g.NB) * g.max_r16 * 128 < 512 << 10)
    while (c > 2 && c * T > 256) --c;
  return c;
}
// Whether the small kernel serves a batch above LS_MAX_T rows over planned groups
// of 16 rows, or the tile kernels do. It reads an adapter again for each group,
// but has fewer steps than they, whose cost goes by tiles of 128 rows, however
// few there are in one. So it takes a batch whose groups run in one wave of
// small clusters, and one whose adapters have few rows, the fewer the larger
// the rank (above 64 it has one CTA an SM). Measured at 6144x6144, small against
// tiles: 260 rows of 64 adapters, rank 64: 22.5, 51.5 us; 1536 of 8, rank 64: 39.3,
// 40.0; 3000 of 8, rank 16: 42.2, 35.3; 2048 of 64, rank 64: 57.6, 55.8 (704x704:
// 12.1, 21.3); 2048 of 64, rank 32: 46.2, 52.3; 4096 of 256, rank 64: 108, 170;
// rank 128, 1024 of 8: 46.9, 57.9; 1024 of 64: 87.7, 67.5.
inline bool lora_planned_small(const LoraGeom& g, int T, int num_sms) {
  const LoraBatch b = lora_batch(g, T);
  return b.groups <= 0.45 * ls_per_sm(g.max_r16) * num_sms || b.rows * g.max_r16 <= (g.max_r16 <= 64 ? 2200.0 : 1100.0);
}

__device__ __forceinline__ uint32_t ls_cluster_rank() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}
__device__ __forceinline__ float4 ld_cluster_f32x4(const void* p, uint32_t rank) {
  uint32_t a;
  float4 v;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"(smem_u32(p)), "r"(rank));
  asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];" : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w) : "r"(a) : "memory");
  return v;
}
__device__ __forceinline__ void add4(float4& a, const float4& b) {
  a.x += b.x;
  a.y += b.y;
  a.z += b.z;
  a.w += b.w;
}
__device__ __forceinline__ void cluster_arrive() { asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory"); }
__device__ __forceinline__ void cluster_wait() { asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory"); }
__device__ __forceinline__ uint4 ldg16(const void* p) { return __ldg(static_cast<const uint4*>(p)); }

// fp16's exponents are too few for u (x and A of a few 2^-10 each already give
// a u whose low part is a subnormal, and |u| may pass 65504). So there each row
// of u is multiplied by a power of two, exactly, that brings a bound on its
// largest |u| to 2^14 .. 2^15, and the row's scale by the inverse: two values
// then hold every u to 2^-22 of itself or 2^-39 of the bound. Infinities and
// NaN, which any factor leaves as they are, have no part in the bound. Beside
// bf16, which needs none of it, a row of rank 16 takes 3.9 to 4.1 us, 64 rows of 64
// adapters of rank 64, 6144x6144, 14.5 to 15.1 (rank 128: 29.6 to 31.3), and in
// tiles 2300 rows of 5, rank 64, 2048x2048, 28.5 to 30.6, 8192 of 8, rank 64,
// 6144x6144, 72.2 to 73.4 (rank 128: 92.5 to 95.7).
template <int ACT>
constexpr bool ROW_POWERS = ACT == ACT_F16;
// |u|, in bits (which order like the values), as far as it is finite.
__device__ __forceinline__ uint32_t finite_bits(float u) {
  const uint32_t b = __float_as_uint(u) & 0x7FFFFFFFu;
  return b < 0x7F800000u ? b : 0u;
}
// From 2^-112 down the factor stays 2^126, so that its inverse is a normal number.
__device__ __forceinline__ uint32_t row_exponent(uint32_t bound) { return max(bound >> 23, 15u); }
__device__ __forceinline__ float row_power(uint32_t bound) { return __uint_as_float((268u - row_exponent(bound)) << 23); }
// The scale times the inverse power, kept finite and, but for a scale of 0, away
// from 0: beyond either end the products B u that it meets (0, at least 2^-48, at
// most 2^38, or infinite) leave fp16's range to the same side as the exact ones.
__device__ __forceinline__ float row_scale(float scale, uint32_t bound) {
  const float s = fabsf(scale) * __uint_as_float((row_exponent(bound) - 14u) << 23);
  return scale == 0.0f ? 0.0f : copysignf(fminf(fmaxf(s, 1.17549435e-38f), 3.40282347e38f), scale);
}

// u as a sum of two values of the activation type. An infinite u keeps its
// value in the first.
template <int ACT>
__device__ __forceinline__ void split_act(float u, uint16_t* hi, uint16_t* lo) {
  *hi = f32_to_act<ACT>(u);
  const float h = act_f32<ACT>(*hi);
  *lo = isinf(h) ? (uint16_t)0 : f32_to_act<ACT>(u - h);
}

// Shared memory: partial sums [LS_WARPS][LS_TOK][r16], the CTA's sum
// [LS_TOK][r16] (fp32), then u's two parts [LS_TOK][r16 + 8] each.
__host__ __device__ constexpr int ls_smem(int r16) {
  return (LS_WARPS + 1) * LS_TOK * r16 * 4 + 2 * LS_TOK * (r16 + 8) * 2;
}

// The groups of a batch of up to LS_COUNT_T rows, found in every CTA: the rows
// of each adapter counted (counts do not depend on the order of the atomics),
// the counts scanned to the adapters' first groups, and a group's rows picked
// out by their places among its adapter's rows. The plan kernel finds the same
// groups, in the same order, and is a launch to wait for (1111 rows of 32
// adapters of ranks to 48, 6144x2056: 21.2 us with it, 19.6 without; 512 rows of
// 64, rank 16, 2048x2048: 9.7, 7.9; 3000 of 512, rank 16, 6144x6144: 82.7, 85.8).
constexpr int LS_COUNT_T = 2048;
template <bool PLANNED>
struct LsGroups {
  int n[LORA_MAX_SLOTS + 1], first[LORA_MAX_SLOTS + 2], rank[LORA_MAX_SLOTS + 1];  // the last: rows without an adapter
  int found;
  uint16_t of[LS_COUNT_T];  // the rows' adapters

  __device__ __forceinline__ void clear(const LoraParams& p, int tid) {
    for (int g = tid; g <= p.g.slots; g += LS_THREADS) n[g] = 0;
  }
  // A warp's rows, 32 at a time.
  __device__ __forceinline__ int rounds(const LoraParams& p) const { return (p.T + LS_THREADS - 1) / LS_THREADS; }

  // Returns the number of groups. wsum: scratch of LS_WARPS words.
  __device__ __forceinline__ int count(const LoraParams& p, int tid, int* wsum) {
    constexpr int IDS = 8;  // loads in flight together
    const int lane = tid & 31, warp = tid >> 5, G = p.g.slots + 1;
    const int many = rounds(p), t0 = warp * many * 32 + lane;
    for (int r0 = 0; r0 < many; r0 += IDS) {
      int id[IDS];
#pragma unroll
      for (int i = 0; i < IDS; ++i) id[i] = r0 + i < many && t0 + (r0 + i) * 32 < p.T ? __ldg(p.ids + t0 + (r0 + i) * 32) : -1;
      if (r0 == 0) {
        for (int g = tid; g < G; g += LS_THREADS) rank[g] = g < G - 1 ? __ldg(reinterpret_cast<const int*>(p.packed) + g) : 0;
        __syncthreads();
      }
#pragma unroll
      for (int i = 0; i < IDS; ++i) {
        if (r0 + i >= many) break;
        const int t = t0 + (r0 + i) * 32;
        const bool row = t < p.T;
        int g = id[i];
        if (g < -1 || g >= G - 1) set_status(p.status, DEV_BAD_ROUTE);
        if (g < 0 || g >= G - 1 || rank[g] == 0) g = G - 1;
        of[t] = row ? (uint16_t)g : (uint16_t)0xFFFF;
        const int g0 = __shfl_sync(0xffffffffu, g, 0);
        if (__all_sync(0xffffffffu, row && g == g0)) {  // a prompt's rows
          if (lane == 0) atomicAdd(&n[g], 32);
        } else if (row) {
          atomicAdd(&n[g], 1);
        }
      }
    }
    __syncthreads();
    // exclusive scan of the adapters' groups, a run of them a thread
    const int per = (G + LS_THREADS - 1) / LS_THREADS;
    int sum = 0;
    for (int g = tid * per; g < min(G, (tid + 1) * per); ++g) sum += (n[g] + LS_TOK - 1) / LS_TOK;
    int in = sum;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const int a = __shfl_up_sync(0xffffffffu, in, d);
      if (lane >= d) in += a;
    }
    if (lane == 31) wsum[warp] = in;
    __syncthreads();
    int at = in - sum;
    for (int w = 0; w < warp; ++w) at += wsum[w];
    for (int g = tid * per; g < min(G, (tid + 1) * per); ++g) {
      first[g] = at;
      at += (n[g] + LS_TOK - 1) / LS_TOK;
    }
    if (tid == LS_THREADS - 1) first[G] = at;
    __syncthreads();
    return first[G];
  }

  // Group gi: its adapter (or -1), that one's rank, and its rows in tok. cnt:
  // scratch of LS_WARPS words.
  __device__ __forceinline__ void rows_of(const LoraParams& p, int gi, int tid, int* cnt, int* tok, int* a, int* r, int* n_tok) {
    const int lane = tid & 31, warp = tid >> 5, G = p.g.slots + 1;
    for (int g = tid; g < G; g += LS_THREADS)
      if (first[g] <= gi && gi < first[g + 1]) found = g;
    if (tid < LS_TOK) tok[tid] = -1;
    __syncthreads();
    const int g = found, skip = (gi - first[g]) * LS_TOK;
    const int many = rounds(p), t0 = warp * many * 32 + lane;
    int mine = 0;
    for (int i = 0; i < many; ++i) mine += __popc(__ballot_sync(0xffffffffu, of[t0 + i * 32] == g));
    if (lane == 0) cnt[warp] = mine;
    __syncthreads();
    int at = -skip;
    for (int w = 0; w < warp; ++w) at += cnt[w];
    if (mine && at < LS_TOK && at + mine > 0) {
      for (int i = 0; i < many; ++i) {
        const bool same = of[t0 + i * 32] == g;
        const unsigned with = __ballot_sync(0xffffffffu, same);
        const int pos = at + __popc(with & ((1u << lane) - 1u));
        if (same && pos >= 0 && pos < LS_TOK) tok[pos] = t0 + i * 32;
        at += __popc(with);
      }
    }
    __syncthreads();
    *a = g < G - 1 ? g : -1;
    *r = rank[g];
    *n_tok = min(LS_TOK, n[g] - skip);
  }
};
template <>
struct LsGroups<false> {
  __device__ __forceinline__ void clear(const LoraParams&, int) {}
};

// R: the largest padded rank of the set, rounded up to 16, 32, 64 or 128.
// PLANNED: the batch's groups of LS_TOK rows, counted in each CTA or from the
// plan kernel's tiles, are taken in turn by as many clusters as run at once.
template <int ACT, int R, bool PLANNED>
__global__ void __launch_bounds__(LS_THREADS, ls_per_sm(R)) lora_small_kernel(LoraParams p) {
  extern __shared__ __align__(16) uint8_t ls_sm[];
  __shared__ int s_tok[LS_TOK], s_cnt[LS_WARPS];
  __shared__ float s_scale[LS_TOK];  // of the group's rows, where each has a power of two
  __shared__ LsGroups<PLANNED> s_groups;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int cta = (int)ls_cluster_rank(), ctas = gridDim.x;  // one cluster a grid row
  const bool counts = PLANNED && p.T <= LS_COUNT_T;
  if (counts) s_groups.clear(p, tid);
  pdl_wait();
  pdl_trigger();
  const int n0 = cta * p.g.NB / ctas * 64, n1 = min(p.g.N, (cta + 1) * p.g.NB / ctas * 64);
  // base alone, for row t
  auto copy_row = [&](int t) {
    if (p.base == p.out) return;
    for (int n = n0 + tid * 8; n < n1; n += LS_THREADS * 8)
      *reinterpret_cast<uint4*>(p.out + (size_t)t * p.ldout + n) =
          p.base ? *reinterpret_cast<const uint4*>(p.base + (size_t)t * p.ldbase + n) : make_uint4(0, 0, 0, 0);
  };
  int groups = blockIdx.y + 1;
  if constexpr (PLANNED) groups = counts ? s_groups.count(p, tid, s_cnt) : p.meta[1];
  for (int gi = blockIdx.y; gi < groups; gi += gridDim.y) {
    int a, rank, n_tok;
    if constexpr (PLANNED) {
      if (counts) {
        s_groups.rows_of(p, gi, tid, s_cnt, s_tok, &a, &rank, &n_tok);
      } else {
        const int4 ti = p.tiles[gi];
        a = ti.x;
        rank = ti.w;
        n_tok = ti.z;
        if (tid < LS_TOK) s_tok[tid] = tid < n_tok ? p.perm[ti.y + tid] : -1;
        __syncthreads();
      }
      if (a < 0) {
        for (int i = 0; i < n_tok; ++i) copy_row(s_tok[i]);
        __syncthreads();
        continue;
      }
    } else {
      a = lora_slot(p, gi);
      rank = a >= 0 ? reinterpret_cast<const int*>(p.packed)[a] : 0;
      if (rank == 0) {
        copy_row(gi);
        return;
      }
      // The group: T <= LS_MAX_T, so thread j looks at row j.
      const bool same = tid < p.T && p.ids[tid] == a;
      if (__syncthreads_count(same && tid < gi) % LS_TOK != 0) return;
      const unsigned later = __ballot_sync(0xffffffffu, same && tid >= gi);
      if (lane == 0) s_cnt[warp] = __popc(later);
      if (tid < LS_TOK) s_tok[tid] = -1;
      __syncthreads();
      {
        int pos = __popc(later & ((1u << lane) - 1u));
        for (int w = 0; w < warp; ++w) pos += s_cnt[w];
        if (same && tid >= gi && pos < LS_TOK) s_tok[pos] = tid;
      }
      __syncthreads();
      n_tok = 0;
#pragma unroll
      for (int w = 0; w < LS_WARPS; ++w) n_tok += s_cnt[w];
      n_tok = min(n_tok, LS_TOK);
    }
    const float scale = reinterpret_cast<const float*>(p.packed + p.g.scale_off)[a];
    const int r16 = (rank + 15) / 16 * 16;
    const uint8_t* block = p.packed + p.g.block_off + (size_t)a * p.g.block_bytes;
    const uint8_t* btiles = block + p.g.b_off;
    const int g = lane >> 2, q = lane & 3;
    const int ta = s_tok[g], tb = s_tok[g + 8];
    const uint4 zero = make_uint4(0, 0, 0, 0);

    // ---- A x over this CTA's k-blocks, half a block (32 of K) a step, the next
    // step's operands on their way
    float acc[R / 8][4];
#pragma unroll
    for (int j = 0; j < R / 8; ++j)
#pragma unroll
      for (int i = 0; i < 4; ++i) acc[j][i] = 0.0f;
    struct Step {
      uint4 xa, xb, w[R / 8];
    };
    const int h1 = 2 * ((cta + 1) * p.g.KB / ctas);
    auto load_a = [&](int h, Step& s) {
      const int k = h * 32 + q * 8;
      s.xa = (h < h1 && ta >= 0 && k < p.g.K) ? ldg16(p.x + (size_t)ta * p.ldx + k) : zero;
      s.xb = (h < h1 && tb >= 0 && k < p.g.K) ? ldg16(p.x + (size_t)tb * p.ldx + k) : zero;
      const uint8_t* tile = block + (size_t)(h >> 1) * r16 * 128 + g * 128 + ((((h & 1) * 4 + q) ^ g) * 16);
#pragma unroll
      for (int j = 0; j < R / 8; ++j) s.w[j] = (h < h1 && 8 * j < r16) ? ldg16(tile + j * 1024) : zero;
    };
    auto mma_a = [&](const Step& s) {
#pragma unroll
      for (int j = 0; j < R / 8; ++j) {
        if (8 * j < r16) {
          mma_16816<ACT>(acc[j], s.xa.x, s.xb.x, s.xa.y, s.xb.y, s.w[j].x, s.w[j].y);
          mma_16816<ACT>(acc[j], s.xa.z, s.xb.z, s.xa.w, s.xb.w, s.w[j].z, s.w[j].w);
        }
      }
    };
    const int h0 = 2 * (cta * p.g.KB / ctas) + warp;
    if constexpr (R <= 64) {
      Step s0, s1;
      load_a(h0, s0);
      for (int h = h0; h < h1; h += 2 * LS_WARPS) {
        load_a(h + LS_WARPS, s1);
        mma_a(s0);
        load_a(h + 2 * LS_WARPS, s0);
        mma_a(s1);
      }
    } else {
      for (int h = h0; h < h1; h += LS_WARPS) {
        Step s0;
        load_a(h, s0);
        mma_a(s0);
      }
    }

    // ---- B's operands for the first 32 columns: they do not wait for u
    // MMA i takes the tile's packed rows 8 i .. 8 i + 7 of these 32 (lora_b_byte)
    struct Cols {
      uint2 w[R / 16][4];
    };
    auto load_b = [&](int n, Cols& s) {
      const uint8_t* tile = btiles + (size_t)(n >> 6) * r16 * 128 + ((n & 63) + g) * 16 + (q >> 1) * 1024 + (q & 1) * 8;
#pragma unroll
      for (int r = 0; r < R / 16; ++r)  // ranks 16 r + 4 q .. + 3 of this lane
#pragma unroll
        for (int i = 0; i < 4; ++i)
          s.w[r][i] = (n < n1 && 16 * r < r16) ? __ldg(reinterpret_cast<const uint2*>(tile + r * 2048 + i * 128)) : make_uint2(0, 0);
    };
    auto load_base = [&](int n, uint4* y) {
      const int c = n + 8 * q;
      const bool in = p.base && n < n1 && c < p.g.N;
      y[0] = in && ta >= 0 ? *reinterpret_cast<const uint4*>(p.base + (size_t)ta * p.ldbase + c) : zero;
      y[1] = in && tb >= 0 ? *reinterpret_cast<const uint4*>(p.base + (size_t)tb * p.ldbase + c) : zero;
    };
    const int nw = n0 + warp * 32;
    Cols b0;
    uint4 y0[2];
    load_b(nw, b0);
    load_base(nw, y0);

    // ---- the group's u: sums over the CTA's warps, then over the cluster
    float* part = reinterpret_cast<float*>(ls_sm);
    float* sum = part + LS_WARPS * LS_TOK * r16;
    uint16_t* u_hi = reinterpret_cast<uint16_t*>(sum + LS_TOK * r16);
    const int ur = r16 + 8;  // row stride of u: 16-byte rows in different banks
    uint16_t* u_lo = u_hi + LS_TOK * ur;
#pragma unroll
    for (int j = 0; j < R / 8; ++j) {
      if (8 * j < r16) {
        float* d = part + (warp * LS_TOK + g) * r16 + 8 * j + 2 * q;
        if (g < n_tok) *reinterpret_cast<float2*>(d) = make_float2(acc[j][0], acc[j][1]);
        if (g + 8 < n_tok) *reinterpret_cast<float2*>(d + 8 * r16) = make_float2(acc[j][2], acc[j][3]);
      }
    }
    __syncthreads();
    for (int i = 4 * tid; i < n_tok * r16; i += 4 * LS_THREADS) {
      float4 v = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll
      for (int w = 0; w < LS_WARPS; ++w) add4(v, *reinterpret_cast<const float4*>(part + w * LS_TOK * r16 + i));
      *reinterpret_cast<float4*>(sum + i) = v;
    }
    cluster_arrive();
    cluster_wait();
    // Four ranks of a row, from r on: their sums over the cluster (those past the
    // rank, where A's zeros met whatever x held, are 0), and their two parts.
    auto gather = [&](int row, int r, bool in) {
      float4 f[8], v = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll
      for (int c = 0; c < 8; ++c)
        f[c] = in && c < ctas ? ld_cluster_f32x4(sum + row * r16 + r, c) : make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll
      for (int c = 0; c < 8; ++c) add4(v, f[c]);  // the same order in every CTA
      return make_float4(r < rank ? v.x : 0.0f, r + 1 < rank ? v.y : 0.0f, r + 2 < rank ? v.z : 0.0f, r + 3 < rank ? v.w : 0.0f);
    };
    auto put = [&](int row, int r, const float4& v) {
      const float u[4] = {v.x, v.y, v.z, v.w};
      uint16_t hi[4], lo[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) split_act<ACT>(u[e], hi + e, lo + e);
      *reinterpret_cast<uint2*>(u_hi + row * ur + r) = make_uint2(hi[0] | (uint32_t)hi[1] << 16, hi[2] | (uint32_t)hi[3] << 16);
      *reinterpret_cast<uint2*>(u_lo + row * ur + r) = make_uint2(lo[0] | (uint32_t)lo[1] << 16, lo[2] | (uint32_t)lo[3] << 16);
    };
    if constexpr (!ROW_POWERS<ACT>) {
      for (int i = 4 * tid; i < n_tok * r16; i += 4 * LS_THREADS) put(i / r16, i % r16, gather(i / r16, i % r16, true));
    } else {  // a row's lanes side by side in a warp
      constexpr int LANES = R <= 64 ? 16 : 32, ROWS = LS_TOK * LANES / LS_THREADS;
      const int r = tid % LANES * 4;
      float4 u[ROWS];
#pragma unroll
      for (int d = 0; d < ROWS; ++d) {
        const int row = tid / LANES + d * (LS_TOK / ROWS);
        u[d] = gather(row, r, row < n_tok && r < r16);
      }
#pragma unroll
      for (int d = 0; d < ROWS; ++d) {
        const int row = tid / LANES + d * (LS_TOK / ROWS);
        uint32_t bound = max(max(finite_bits(u[d].x), finite_bits(u[d].y)), max(finite_bits(u[d].z), finite_bits(u[d].w)));
        bound = __reduce_max_sync(LANES == 32 ? 0xffffffffu : 0xffffu << (lane & 16), bound);
        const float power = row_power(bound);
        if (r == 0) s_scale[row] = row_scale(scale, bound);
        if (row < n_tok && r < r16) put(row, r, make_float4(power * u[d].x, power * u[d].y, power * u[d].z, power * u[d].w));
      }
    }
    __syncthreads();
    cluster_arrive();  // this CTA has read the others' sums

    // ---- B u over this CTA's columns, 32 a step (rows of u past n_tok are not
    // set; they meet no other row, and their results are not stored)
    const float by[2] = {ROW_POWERS<ACT> ? s_scale[g] : scale, ROW_POWERS<ACT> ? s_scale[g + 8] : scale};
    auto mma_b = [&](int n, const Cols& s, uint4* y) {
      float d[4][4];
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int e = 0; e < 4; ++e) d[i][e] = 0.0f;
#pragma unroll
      for (int r = 0; r < R / 16; ++r) {
        if (16 * r < r16) {
          const int o = 16 * r + 4 * q;
          const uint2 ha = *reinterpret_cast<const uint2*>(u_hi + g * ur + o);
          const uint2 hb = *reinterpret_cast<const uint2*>(u_hi + (g + 8) * ur + o);
          const uint2 la = *reinterpret_cast<const uint2*>(u_lo + g * ur + o);
          const uint2 lb = *reinterpret_cast<const uint2*>(u_lo + (g + 8) * ur + o);
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            mma_16816<ACT>(d[i], ha.x, hb.x, ha.y, hb.y, s.w[r][i].x, s.w[r][i].y);
            mma_16816<ACT>(d[i], la.x, lb.x, la.y, lb.y, s.w[r][i].x, s.w[r][i].y);
          }
        }
      }
      const int c = n + 8 * q;
      if (c < p.g.N) {
#pragma unroll
        for (int half = 0; half < 2; ++half) {
          const int t = half ? tb : ta;
          if (t < 0) continue;
          uint32_t* yw = reinterpret_cast<uint32_t*>(&y[half]);
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const float2 b = act_x2_to_f32<ACT>(yw[i]);
            yw[i] = f32_to_act_x2<ACT>(fmaf(by[half], d[i][2 * half], b.x), fmaf(by[half], d[i][2 * half + 1], b.y));
          }
          *reinterpret_cast<uint4*>(p.out + (size_t)t * p.ldout + c) = y[half];
        }
      }
    };
    if constexpr (R <= 64) {
      Cols b1;
      uint4 y1[2];
      for (int n = nw; n < n1; n += 2 * LS_WARPS * 32) {
        load_b(n + LS_WARPS * 32, b1);
        load_base(n + LS_WARPS * 32, y1);
        mma_b(n, b0, y0);
        if (n + LS_WARPS * 32 >= n1) break;
        load_b(n + 2 * LS_WARPS * 32, b0);
        load_base(n + 2 * LS_WARPS * 32, y0);
        mma_b(n + LS_WARPS * 32, b1, y1);
      }
    } else {
      for (int n = nw; n < n1; n += LS_WARPS * 32) {
        mma_b(n, b0, y0);
        load_b(n + LS_WARPS * 32, b0);
        load_base(n + LS_WARPS * 32, y0);
      }
    }
    cluster_wait();  // the others have read this CTA's sums
  }
}

// One cluster a grid row; PLANNED: the groups are in the plan, and as many
// clusters as run at once take them.
template <int ACT, int R, bool PLANNED>
static cudaError_t small_as(const LoraParams& p, cudaStream_t st) {
  static std::atomic<unsigned long long> done{0};
  cudaError_t e = ensure_smem_attr(lora_small_kernel<ACT, R, PLANNED>, ls_smem(R), done);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.blockDim = dim3(LS_THREADS);
  cfg.dynamicSmemBytes = (size_t)ls_smem(R);
  cfg.stream = st;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  // How many clusters of each size run at once, asked once.
  static std::atomic<int> known[LS_MAX_CLUSTER + 1];
  int fits[LS_MAX_CLUSTER + 1] = {};
  for (unsigned c = 2; c <= LS_MAX_CLUSTER; ++c) {
    fits[c] = known[c].load(std::memory_order_relaxed);
    if (fits[c] > 0) continue;
    attr[1].val.clusterDim = {c, 1, 1};
    cfg.gridDim = dim3(c);
    e = cudaOccupancyMaxActiveClusters(&fits[c], lora_small_kernel<ACT, R, PLANNED>, &cfg);
    if (e != cudaSuccess) return e;
    fits[c] = fits[c] < 1 ? 1 : fits[c];
    known[c].store(fits[c], std::memory_order_relaxed);
  }
  const unsigned ctas = (unsigned)ls_cluster(p.g, p.T, fits);
  attr[1].val.clusterDim = {ctas, 1, 1};
  cfg.gridDim = dim3(ctas, PLANNED ? (unsigned)fits[ctas] : (unsigned)p.T);
  count_launches(1);
  return cudaLaunchKernelEx(&cfg, lora_small_kernel<ACT, R, PLANNED>, p);
}
template <int ACT, bool PLANNED>
static cudaError_t small_of(const LoraParams& p, cudaStream_t st) {
  if (p.g.max_r16 <= 16) return small_as<ACT, 16, PLANNED>(p, st);
  if (p.g.max_r16 <= 32) return small_as<ACT, 32, PLANNED>(p, st);
  if (p.g.max_r16 <= 64) return small_as<ACT, 64, PLANNED>(p, st);
  return small_as<ACT, 128, PLANNED>(p, st);
}

// ------------------------------------------------------------ larger batches: plan, A x, B u
// Three launches. The plan groups the rows by adapter and cuts the groups into
// tiles of up to 128 rows; the rows of a tile sit on the M side of tcgen05.mma
// and the adapter on its N side. 8192 rows of 12 requests, ranks up to 64,
// 6144x6144 take 72.3 us, about 5 for the plan, 22 for A x (104 MB, 70% of HBM
// with its start and end) and 45 for B u (201 MB, 67%); the floor is 46.

// One CTA. Rows without an adapter (or with an empty slot) form the last group.
// The rows of a group keep their order, so that the tiles, and with them the
// order of every sum, depend on the ids alone: each warp counts its own range
// of rows (s_base[warp][group]), and the counts are summed over the warps.
// The loops are kept rolled: the kernel runs once through its code, and what
// it costs is mostly latency, of instruction fetches too.
constexpr int LP_THREADS = 1024;
constexpr int LP_WARPS = LP_THREADS / 32;
constexpr int LP_IDS = 8;
constexpr int LP_ROWS = 8192;  // rows whose words fit shared memory; of a larger batch they are kept in the u scratch
constexpr int lp_smem(int slots) { return (LP_ROWS + LP_WARPS * (slots + 1)) * 4; }
__global__ void __launch_bounds__(LP_THREADS) lora_plan_kernel(LoraParams p) {
  extern __shared__ int s_word[];  // [LP_ROWS]: group, and place << 10 in the warp's part of it
  __shared__ int s_rank[LORA_MAX_SLOTS + 1], s_wsum[2][LP_WARPS];
  static_assert(LORA_MAX_SLOTS + 1 <= 1 << 10 && LORA_MAX_SLOTS + 1 <= LP_THREADS, "group bits");
  static_assert(LORA_MAX_ROWS / LP_WARPS <= 1 << 21 && LORA_MAX_ROWS % LP_THREADS == 0, "place bits, the sign left out");
  int* s_base = s_word + LP_ROWS;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int G = p.g.slots + 1;
  for (int i = tid; i < LP_WARPS * G; i += LP_THREADS) s_base[i] = 0;
  pdl_wait();
  pdl_trigger();
  const int rounds = (p.T + LP_THREADS - 1) / LP_THREADS;  // 32 rows of the warp's range each
  const int t0 = warp * rounds * 32 + lane;
  int* word = p.T <= LP_ROWS ? s_word : reinterpret_cast<int*>(p.u);
  int* mine = s_base + warp * G;
  if (p.bound)
    for (int t = tid; t < p.T; t += LP_THREADS) p.bound[t] = 0u;
  if (tid < G) s_rank[tid] = tid < p.g.slots ? __ldcg(reinterpret_cast<const int*>(p.packed) + tid) : 0;
  int bits = 1;  // of a group's number
  while (G > 1 << bits) ++bits;
  for (int r0 = 0; r0 < rounds; r0 += LP_IDS) {
    int id[LP_IDS];  // loads in flight together
#pragma unroll
    for (int i = 0; i < LP_IDS; ++i) id[i] = t0 + (r0 + i) * 32 < p.T ? __ldcg(p.ids + t0 + (r0 + i) * 32) : -2;
    if (r0 == 0) __syncthreads();
#pragma unroll
    for (int i = 0; i < LP_IDS; ++i) {
      if (r0 + i >= rounds) break;
      int g = id[i];
      const bool row = t0 + (r0 + i) * 32 < p.T;
      if (row && (g < -1 || g >= p.g.slots)) set_status(p.status, DEV_BAD_ROUTE);
      if (g < 0 || g >= p.g.slots || s_rank[g] == 0) g = G - 1;
      // the lanes with this lane's group, bit by bit
      unsigned peers = __ballot_sync(0xffffffffu, row);
      const int g0 = __shfl_sync(0xffffffffu, g, 0);
      const int most = __all_sync(0xffffffffu, !row || g == g0) ? 0 : bits;  // often all the same
#pragma unroll 1
      for (int b = 0; b < most; ++b) {
        const bool one = (g >> b) & 1;
        const unsigned with = __ballot_sync(0xffffffffu, one);
        peers &= one ? with : ~with;
      }
      const int place = mine[g] + __popc(peers & ((1u << lane) - 1u));
      __syncwarp();
      if (row && lane == __ffs(peers) - 1) mine[g] += __popc(peers);
      if (row) word[t0 + (r0 + i) * 32] = g | place << 10;
      __syncwarp();
    }
  }
  __syncthreads();
  // Each group's counts become the warps' places in it: warp w takes the
  // groups w, w + 32, .., lane = warp counted.
  __shared__ int s_n[LORA_MAX_SLOTS + 1], s_tile[LORA_MAX_SLOTS + 2];
#pragma unroll 1
  for (int g = warp; g < G; g += LP_WARPS) {
    const int c = s_base[lane * G + g];
    int in = c;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const int a = __shfl_up_sync(0xffffffffu, in, d);
      if (lane >= d) in += a;
    }
    s_base[lane * G + g] = in - c;
    if (lane == 31) s_n[g] = in;
  }
  __syncthreads();
  // Exclusive scans of the groups' rows and tiles.
  const int n = tid < G ? s_n[tid] : 0, nt = (n + p.tile_rows - 1) / p.tile_rows;
  int in = n, it = nt;
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const int a = __shfl_up_sync(0xffffffffu, in, d), b = __shfl_up_sync(0xffffffffu, it, d);
    if (lane >= d) {
      in += a;
      it += b;
    }
  }
  if (lane == 31) {
    s_wsum[0][warp] = in;
    s_wsum[1][warp] = it;
  }
  __syncthreads();
  int row0 = in - n, tile0 = it - nt;
#pragma unroll 1
  for (int w = 0; w < warp && warp * 32 < G; ++w) {
    row0 += s_wsum[0][w];
    tile0 += s_wsum[1][w];
  }
  __syncthreads();
  if (tid < G) {
    s_n[tid] = row0;  // from here on: where the group starts
    s_tile[tid] = tile0;
  }
  if (tid == G - 1) {
    s_tile[G] = tile0 + nt;
    p.meta[0] = tile0;
    p.meta[1] = tile0 + nt;
  }
  __syncthreads();
  for (int j = tid; j < s_tile[G]; j += LP_THREADS) {
    int lo = 0, hi = G - 1;  // the last group that starts at or before tile j
    while (lo < hi) {
      const int mid = (lo + hi + 1) >> 1;
      if (s_tile[mid] <= j) lo = mid;
      else hi = mid - 1;
    }
    const int first = s_n[lo] + (j - s_tile[lo]) * p.tile_rows, end = lo < G - 1 ? s_n[lo + 1] : p.T;
    p.tiles[j] = make_int4(lo < G - 1 ? lo : -1, first, min(p.tile_rows, end - first), s_rank[lo]);
  }
#pragma unroll 2
  for (int r = 0; r < rounds; ++r) {
    const int t = t0 + r * 32;
    if (t < p.T) {
      const int w = word[t], g = w & 1023;
      p.perm[s_n[g] + mine[g] + (w >> 10)] = t;
    }
  }
}

// ------------------------------------------------------------ the tile kernels
// Both kernels run one persistent CTA per SM over a contiguous share of the
// batch's units (64 of K, or 64 columns, of a tile), so that every SM has the
// same number of units whatever the tiles are. Their warps have roles: some
// bring tiles into a ring, one issues the MMAs, the others turn accumulators
// into results.
constexpr int LT_X_BYTES = LORA_TILE_ROWS * 128;  // 128 rows x 64 values
constexpr int LT_SMEM = 232448 - 1024 - 2048;     // a CTA's shared memory without alignment and barriers
constexpr int LT_MAX_STAGES = 8;

// What a tile's unit range needs.
struct LoraTile {
  int adapter, pos, n, rank, r16;
  const uint8_t* block;
};
__device__ __forceinline__ LoraTile lora_tile(const LoraParams& p, int tile) {
  const int4 ti = __ldcg(p.tiles + tile);
  LoraTile t;
  t.adapter = ti.x;
  t.pos = ti.y;
  t.n = ti.z;
  t.rank = ti.w;
  t.r16 = (t.rank + 15) / 16 * 16;
  t.block = p.packed + p.g.block_off + (size_t)(ti.x >= 0 ? ti.x : 0) * p.g.block_bytes;
  return t;
}
// Ring position: slot and the parity of its current use.
struct RingPos {
  int slot = 0;
  uint32_t ph = 0;
  __device__ __forceinline__ void next(int stages) {
    if (++slot == stages) {
      slot = 0;
      ph ^= 1u;
    }
  }
  __device__ __forceinline__ void back(int stages) {
    if (--slot < 0) {
      slot = stages - 1;
      ph ^= 1u;
    }
  }
};

__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src, uint32_t bytes) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(bytes) : "memory");
}
__device__ __forceinline__ void cp_async_wait_all() { asm volatile("cp.async.wait_all;" ::: "memory"); }
// This thread's arrival on the barrier, once all its copies so far have landed.
__device__ __forceinline__ void cp_async_arrive(uint64_t* bar) {
  asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(smem_u32(bar)) : "memory");
}

// Four producer warps bring 128 rows x 128 bytes (64 values of each row) and
// one adapter tile into each ring slot. The rows of a tile lie anywhere, so
// they come by 16-byte cp.async, 8 a thread, into the 128-byte swizzled layout
// that the tensor cores read. (TMA gathers of four rows took about 1.4 us for
// the 128 rows, twice what HBM needs for them.) The copies themselves arrive on
// the slot's barrier: announcing a slot from the producer some slots later
// leaves the consumers as many slots less to hide the hand-over in (measured
// with 6 slots announced 5 behind: 84 against 40 us for B u at 8192 rows).
constexpr int LT_PROD_WARPS = 4;
constexpr int LT_FULL_COUNT = LT_PROD_WARPS * 32 + 1;  // and the adapter tile's expected bytes
struct LoraProducer {
  uint8_t* ring;
  uint64_t *full, *empty;
  int stages, stage_bytes, tid;
  volatile int* abort;
  uint64_t lim;
  RingPos at;
  int issued = 0;
  const uint16_t* src[8];

  // Rows tid / 8 + 16 j of the tile, chunk tid % 8.
  __device__ __forceinline__ void rows(const LoraParams& p, const LoraTile& t, const uint16_t* x, size_t ld) {
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const int r = (tid >> 3) + 16 * j;
      src[j] = x && r < t.n ? x + (size_t)__ldcg(p.perm + t.pos + r) * ld + (tid & 7) * 8 : nullptr;
    }
  }
  // One unit: columns col .. col + 63 of width (zeros past it), and w_bytes of the adapter.
  __device__ __forceinline__ bool fill(int col, int width, const uint8_t* w, uint32_t w_bytes) {
    if (!__all_sync(0xffffffffu, mbar_wait(&empty[at.slot], at.ph ^ 1u, abort, lim))) return false;
    uint8_t* st = ring + at.slot * stage_bytes;
    if (tid < 32) {
      mbar_expect_tx_elect(&full[at.slot], w_bytes);
      bulk_g2s_if(tid == 0 && w_bytes > 0, st + LT_X_BYTES, w, w_bytes, &full[at.slot]);
    }
    const bool in = col + (tid & 7) * 8 < width;
    const uint32_t dst = smem_u32(st) + (tid >> 3) * 128 + (((tid & 7) ^ ((tid >> 3) & 7)) * 16);
    const int at_col = in ? col : -(tid & 7) * 8;  // past the width: zeros, and a source inside the row
#pragma unroll
    for (int j = 0; j < 8; ++j)
      if (src[j]) cp_async16(dst + j * 2048, src[j] + at_col, in ? 16u : 0u);
    cp_async_arrive(&full[at.slot]);
    at.next(stages);
    ++issued;
    return true;
  }
  // After a wait gave up: the copies in flight are waited for (bounded).
  __device__ __forceinline__ void drain() {
    cp_async_wait_all();
    volatile int never = 0;
    for (int b = 0; b < stages && b < issued; ++b) {
      at.back(stages);
      mbar_wait(&full[at.slot], at.ph, &never, lim);
    }
  }
};

// Warp roles of the A x kernel: 0..3 producers, 4..7 epilogue, 8 MMA.
constexpr int LA_THREADS = 288;
__host__ __device__ constexpr int la_stages(int r16) {
  return LT_SMEM / (LT_X_BYTES + r16 * 128) < LT_MAX_STAGES ? LT_SMEM / (LT_X_BYTES + r16 * 128) : LT_MAX_STAGES;
}
__host__ __device__ constexpr int la_smem(int r16) { return 1024 + la_stages(r16) * (LT_X_BYTES + r16 * 128); }
// At least this many units a CTA, so that few pieces of a tile have to be joined.
constexpr int LA_MIN_UNITS = 4;
// The shares of A x: U units over G CTAs, in order. A tile whose K
// extent lies in several shares is summed in pieces, at most two of a CTA's
// own: the end of a tile that another began (piece slot 2 b), and the
// beginning of one (2 b + 1).
// All counts fit 32 bits: a unit stands for up to 128 x 64 values.
struct LoraShares {
  unsigned U, G, q, r;  // the first r CTAs have q + 1 units, the others q
  __device__ __forceinline__ LoraShares(unsigned units, unsigned ctas) : U(units), G(ctas), q(units / ctas), r(units % ctas) {}
  __device__ __forceinline__ unsigned begin(unsigned b) const { return b < G ? q * b + min(b, r) : U; }
  __device__ __forceinline__ unsigned cta(unsigned v) const {
    return v < r * (q + 1) ? v / (q + 1) : r + (v - r * (q + 1)) / q;
  }
};
__device__ __forceinline__ LoraShares shrink_shares(const LoraParams& p) {
  const unsigned U = (unsigned)__ldcg(p.meta) * (unsigned)p.g.KB;
  return LoraShares(U, min(gridDim.x, max(1u, U / LA_MIN_UNITS)));
}
// The part of a share that lies in one tile: n units from `first` of `per`.
struct LoraSpan {
  int tile, first, n;
  __device__ __forceinline__ LoraSpan(unsigned v, unsigned v1, unsigned per)
      : tile((int)(v / per)), first((int)(v % per)), n((int)min(v1 - v, per - v % per)) {}
};

// A x of a tile's rows: to u[pos][r] where a CTA has the tile's whole K extent,
// else a sum for each piece to part[slot][row][r], which the reader adds up
// (letting the last CTA of a tile add them up here cost 10 us of this kernel's
// tail at 8192 rows). For fp16 also a bound on each row's |u|, to bound[pos]:
// the row's largest, or its pieces' largest times their number. HBM bounds it:
// 16 KB of x a unit, four MMAs of 128 x r x 16.
template <int ACT>
__global__ void __launch_bounds__(LA_THREADS, 1)
    lora_shrink_kernel(const __grid_constant__ LoraParams p) {
  extern __shared__ uint8_t lt_sm[];
  __shared__ __align__(8) uint64_t full[LT_MAX_STAGES], empty[LT_MAX_STAGES], acc_full[2], acc_empty[2], mma_done;
  __shared__ uint32_t s_tmem;
  __shared__ int s_abort;
  uint8_t* smem = lt_sm + ((1024u - (smem_u32(lt_sm) & 1023u)) & 1023u);
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int stages = la_stages(p.g.max_r16);
  const int stage_bytes = LT_X_BYTES + p.g.max_r16 * 128;
  const uint32_t acc_cols = p.g.max_r16 <= 32 ? 32u : (p.g.max_r16 <= 64 ? 64u : 128u);
  if (warp == 8) {
    tmem_alloc(&s_tmem, 2 * acc_cols);
    tmem_relinquish();
  }
  if (tid == 0) {
    for (int i = 0; i < stages; ++i) {
      mbar_init(&full[i], LT_FULL_COUNT);
      mbar_init(&empty[i], 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&acc_full[i], 1);
      mbar_init(&acc_empty[i], 4);
    }
    mbar_init(&mma_done, 1);
    fence_mbar_init();
    s_abort = 0;
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = s_tmem;
  pdl_wait();
  pdl_trigger();  // after the TMEM allocation: the next kernel's may then wait for this one's end
  volatile int* abort = &s_abort;
  const uint64_t lim = p.wait_limit_ns;
  const LoraShares shares = shrink_shares(p);
  const unsigned v0 = shares.begin(blockIdx.x), v1 = shares.begin(blockIdx.x + 1);

  if (warp < LT_PROD_WARPS) {
    LoraProducer pr{smem, full, empty, stages, stage_bytes, tid, abort, lim};
    bool ok = true;
    for (unsigned v = v0; v < v1 && ok;) {
      const LoraSpan sp(v, v1, p.g.KB);
      const int kb0 = sp.first, nk = sp.n;
      const LoraTile t = lora_tile(p, sp.tile);
      v += nk;
      pr.rows(p, t, p.x, p.ldx);
      const uint32_t a_bytes = (uint32_t)t.r16 * 128;
      for (int i = kb0; i < kb0 + nk && ok; ++i) ok = pr.fill(i * 64, p.g.K, t.block + (size_t)i * a_bytes, a_bytes);
    }
    if (!ok) {
      if (lane == 0) {
        s_abort = 1;
        set_status(p.status, DEV_TIMEOUT);
      }
      pr.drain();
    }
  } else if (warp == 8) {
    RingPos rp;
    bool ok = true;
    int j = 0;
    for (unsigned v = v0; v < v1 && ok; ++j) {
      const LoraSpan sp(v, v1, p.g.KB);
      const int nk = sp.n;
      const LoraTile t = lora_tile(p, sp.tile);
      v += nk;
      const int buf = j & 1;
      ok = __all_sync(0xffffffffu, mbar_wait(&acc_empty[buf], ((uint32_t)(j >> 1) & 1u) ^ 1u, abort, lim));
      tc_fence_after();
      const uint32_t idesc = idesc_kf16<ACT>(128, t.r16), d = tmem + (uint32_t)buf * acc_cols;
      for (int i = 0; i < nk && ok; ++i) {
        if (!__all_sync(0xffffffffu, mbar_wait(&full[rp.slot], rp.ph, abort, lim))) {
          ok = false;
          break;
        }
        fence_async_smem();  // the rows came through the generic proxy
        const uint32_t x_lo = smem_desc_sw128_lo(smem_u32(smem + rp.slot * stage_bytes));
        const uint32_t a_lo = x_lo + (LT_X_BYTES >> 4);
#pragma unroll
        for (int ks = 0; ks < 4; ++ks)
          umma_kf16_warp(d, desc_from_lo(x_lo + 2 * ks), desc_from_lo(a_lo + 2 * ks), idesc, (i | ks) ? 1u : 0u);
        umma_commit_warp(&empty[rp.slot]);
        rp.next(stages);
      }
      if (ok) umma_commit_warp(&acc_full[buf]);
    }
    if (!ok && lane == 0) {
      s_abort = 1;
      set_status(p.status, DEV_TIMEOUT);
    }
    umma_commit_warp(&mma_done);  // drain the MMAs before TMEM is released
    volatile int never = 0;
    mbar_wait(&mma_done, 0, &never, lim);
  } else {
    const int row = (warp & 3) * 32 + lane;
    int j = 0;
    for (unsigned v = v0; v < v1; ++j) {
      const LoraSpan sp(v, v1, p.g.KB);
      const int kb0 = sp.first, nk = sp.n;
      const LoraTile t = lora_tile(p, sp.tile);
      v += nk;
      const int buf = j & 1;
      if (!__all_sync(0xffffffffu, mbar_wait(&acc_full[buf], (uint32_t)(j >> 1) & 1u, abort, lim))) {
        if (lane == 0) {
          s_abort = 1;
          set_status(p.status, DEV_TIMEOUT);
        }
        break;
      }
      tc_fence_after();
      // lane = row
      float* dst = nk == p.g.KB ? p.u + (size_t)(t.pos + row) * p.g.max_r16
                                : p.part + ((size_t)(2 * blockIdx.x + (kb0 == 0)) * LORA_TILE_ROWS + row) * p.g.max_r16;
      uint32_t bound = 0;
      for (int col = 0; col < t.r16; col += 16) {
        uint32_t w[16];
        tmem_ld16(tmem + ((uint32_t)((warp & 3) * 32) << 16) + (uint32_t)buf * acc_cols + col, w);
        tmem_wait_ld();
        if constexpr (ROW_POWERS<ACT>) {
#pragma unroll
          for (int i = 0; i < 16; ++i) bound = max(bound, finite_bits(__uint_as_float(w[i])));
        }
        if (row < t.n) {
#pragma unroll
          for (int i = 0; i < 4; ++i)
            *reinterpret_cast<uint4*>(dst + col + 4 * i) = make_uint4(w[4 * i], w[4 * i + 1], w[4 * i + 2], w[4 * i + 3]);
        }
      }
      if constexpr (ROW_POWERS<ACT>) {
        const unsigned w0 = (unsigned)sp.tile * (unsigned)p.g.KB;
        const unsigned pieces = shares.cta(w0 + p.g.KB - 1) - shares.cta(w0) + 1;
        const float most = fminf(__uint_as_float(bound) * (float)pieces, 3.40282347e38f);
        if (row < t.n) atomicMax(p.bound + t.pos + row, __float_as_uint(most));  // in any order the same
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&acc_empty[buf]);
    }
  }
  __syncwarp();
  tc_fence_before();
  __syncthreads();
  if (warp == 8) {
    tc_fence_after();
    tmem_dealloc(tmem, 2 * acc_cols);
  }
}

// Warp roles of the B u kernel: 0 producer, 1 MMA, 2..7 u operand, 8..23
// epilogue (two groups of 8, which take alternate units).
constexpr int LB_THREADS = 768;
constexpr int LB_WARP_U = 2, LB_WARP_EPI = 8;
constexpr int LB_U_WARPS = LB_WARP_EPI - LB_WARP_U, LB_EPI_WARPS = 8;  // epilogue warps of a group
constexpr int LB_FIRST_WARPS = LB_U_WARPS + 2 * LB_EPI_WARPS;           // warps that form the first u
constexpr int LB_ACC = 4;     // accumulators of 64 columns
constexpr int LB_MAX_STAGES = 12;  // B tiles in the ring
__host__ __device__ constexpr int lb_u_bytes(int r16) { return 2 * LORA_TILE_ROWS * r16 * 2; }
// u's two parts are held twice, so that the next tile's are ready in time;
// above rank 80 once, which leaves the room to the ring.
__host__ __device__ constexpr int lb_u_bufs(int r16) { return r16 <= 80 ? 2 : 1; }
__host__ __device__ constexpr int lb_stages(int r16) {
  return (LT_SMEM - lb_u_bufs(r16) * lb_u_bytes(r16)) / (r16 * 128) < LB_MAX_STAGES
             ? (LT_SMEM - lb_u_bufs(r16) * lb_u_bytes(r16)) / (r16 * 128)
             : LB_MAX_STAGES;
}
__host__ __device__ constexpr int lb_smem(int r16) {
  return 1024 + lb_u_bufs(r16) * lb_u_bytes(r16) + lb_stages(r16) * r16 * 128;
}
static_assert(lb_stages(64) == LB_MAX_STAGES && lb_stages(96) >= 2 && lb_stages(LORA_MAX_RANK) >= 5, "stages");
static_assert(LB_ACC % 2 == 0, "each epilogue group has accumulators of its own");

// u of one tile as the A operand, in its two parts: 16-byte core-matrix rows,
// [r16 / 8][128 rows]. The sums of the pieces are added up in K order. Warp w of
// nw; a lane takes 4 ranks of one row, a warp 8 rows of 16 ranks, Q such at once
// (loads in flight together: the walk over the pieces is latency alone).
struct LoraPieces {
  const float* first;
  const float* more;  // the second piece
  const uint32_t* bound;  // of the rows, where each has a power of two
  int n;
};
template <int ACT, int Q>
__device__ __forceinline__ void lora_u_operand(const LoraTile& t, const LoraPieces& pc, int max_r16, uint8_t* hi, int w,
                                               int nw, int lane) {
  uint8_t* lo = hi + LORA_TILE_ROWS * t.r16 * 2;
  const size_t step = (size_t)2 * LORA_TILE_ROWS * max_r16;
  const int items = (t.r16 / 16) * (LORA_TILE_ROWS / 8);
  for (int i0 = w; i0 < items; i0 += Q * nw) {
    float4 f[Q];
    int row[Q], k[Q];
    bool in[Q];
#pragma unroll
    for (int q = 0; q < Q; ++q) {
      const int i = i0 + q * nw;
      row[q] = (i & 15) * 8 + (lane >> 2);
      k[q] = (i >> 4) * 16 + (lane & 3) * 4;
      in[q] = i < items && row[q] < t.n;
      f[q] = in[q] ? __ldcg(reinterpret_cast<const float4*>(pc.first + (size_t)row[q] * max_r16 + k[q]))
                   : make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    }
    for (int b = 0; b < pc.n - 1; ++b) {
      float4 m[Q];
#pragma unroll
      for (int q = 0; q < Q; ++q) {
        m[q] = in[q] ? __ldcg(reinterpret_cast<const float4*>(pc.more + b * step + (size_t)row[q] * max_r16 + k[q]))
                     : make_float4(0.0f, 0.0f, 0.0f, 0.0f);
      }
#pragma unroll
      for (int q = 0; q < Q; ++q)
        f[q] = make_float4(f[q].x + m[q].x, f[q].y + m[q].y, f[q].z + m[q].z, f[q].w + m[q].w);
    }
    uint32_t bound[Q];  // asked for here: with the sums above it would be waited for before the walk
    if constexpr (ROW_POWERS<ACT>) {
#pragma unroll
      for (int q = 0; q < Q; ++q) bound[q] = in[q] ? __ldcg(pc.bound + row[q]) : 0u;
    }
#pragma unroll
    for (int q = 0; q < Q; ++q) {
      if (i0 + q * nw >= items) break;
      const float power = ROW_POWERS<ACT> ? row_power(bound[q]) : 1.0f;
      float v[4] = {f[q].x, f[q].y, f[q].z, f[q].w};
      if constexpr (ROW_POWERS<ACT>) {
#pragma unroll
        for (int j = 0; j < 4; ++j) v[j] *= power;
      }
      uint16_t h[4], l[4];
      // past the rank A's zeros met whatever x held
#pragma unroll
      for (int j = 0; j < 4; ++j) split_act<ACT>(k[q] + j < t.rank ? v[j] : 0.0f, &h[j], &l[j]);
      const int at = ((k[q] >> 3) * LORA_TILE_ROWS + row[q]) * 16 + (k[q] & 4) * 2;
      *reinterpret_cast<uint2*>(hi + at) = make_uint2(h[0] | (uint32_t)h[1] << 16, h[2] | (uint32_t)h[3] << 16);
      *reinterpret_cast<uint2*>(lo + at) = make_uint2(l[0] | (uint32_t)l[1] << 16, l[2] | (uint32_t)l[3] << 16);
    }
  }
}
__device__ __forceinline__ LoraPieces lora_pieces(const LoraParams& p, const LoraShares& ks, int tile, const LoraTile& t) {
  const unsigned w0 = (unsigned)tile * (unsigned)p.g.KB;
  const unsigned b0 = ks.cta(w0), b1 = ks.cta(w0 + p.g.KB - 1);
  LoraPieces pc;
  pc.n = (int)(b1 - b0) + 1;
  pc.first = b0 == b1 ? p.u + (size_t)t.pos * p.g.max_r16
                      : p.part + (size_t)(2 * b0 + 1) * LORA_TILE_ROWS * p.g.max_r16;
  pc.more = p.part + (size_t)(2 * b0 + 2) * LORA_TILE_ROWS * p.g.max_r16;
  pc.bound = p.bound + t.pos;
  return pc;
}

// (a, b) * s + (c, d), both halves in one instruction.
__device__ __forceinline__ float2 fma_x2(float a, float b, float s, float2 c) {
  float2 r;
  asm("{\n\t.reg .b64 x, y, z, w;\n\t"
      "mov.b64 x, {%2, %3};\n\tmov.b64 y, {%4, %4};\n\tmov.b64 z, {%5, %6};\n\t"
      "fma.rn.f32x2 w, x, y, z;\n\tmov.b64 {%0, %1}, w;\n\t}"
      : "=f"(r.x), "=f"(r.y)
      : "f"(a), "f"(b), "f"(s), "f"(c.x), "f"(c.y));
  return r;
}

// out = base + scale B u. u enters as its two parts (split_act), whose products
// with B add up in the same accumulator. An epilogue warp owns 32 rows and 32
// columns of every second unit; a lane holds 16 bytes of 4 rows, whose base
// values it has loaded two units ahead. It moves 16 KB of base in and of out a
// unit, at 67% of HBM (8192 rows): its start and tail on 152 SMs and the epilogue
// warps' issue of loads and stores take the rest. Without B's permuted rows the results had to cross shared memory
// to reach 64 bytes of a row together: 54 against 44 us at 8192 rows.
template <int ACT>
__global__ void __launch_bounds__(LB_THREADS, 1) lora_expand_kernel(const __grid_constant__ LoraParams p) {
  extern __shared__ uint8_t lt_sm[];
  __shared__ __align__(8) uint64_t full[LB_MAX_STAGES], empty[LB_MAX_STAGES], acc_full[LB_ACC], acc_empty[LB_ACC], u_full[2],
      u_empty[2], mma_done;
  __shared__ uint32_t s_tmem;
  __shared__ int s_abort;
  uint8_t* smem = lt_sm + ((1024u - (smem_u32(lt_sm) & 1023u)) & 1023u);
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int u_bytes = lb_u_bytes(p.g.max_r16), u_bufs = lb_u_bufs(p.g.max_r16);
  const int stage_bytes = p.g.max_r16 * 128, stages = lb_stages(p.g.max_r16);
  uint8_t* ring = smem + u_bufs * u_bytes;
  if (warp == 1) {
    tmem_alloc(&s_tmem, LB_ACC * 64);
    tmem_relinquish();
  }
  if (tid == 0) {
    for (int i = 0; i < stages; ++i) {
      mbar_init(&full[i], 1);
      mbar_init(&empty[i], 1);
    }
    for (int i = 0; i < LB_ACC; ++i) {
      mbar_init(&acc_full[i], 1);
      mbar_init(&acc_empty[i], LB_EPI_WARPS);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&u_full[i], LB_U_WARPS);
      mbar_init(&u_empty[i], 1);
    }
    mbar_init(&mma_done, 1);
    fence_mbar_init();
    s_abort = 0;
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = s_tmem;
  // Only the warps that read u wait for the A x kernel. The others read what
  // was complete before that kernel's own wait returned, which is before any
  // CTA of this one may start: the plan, the base and the adapters (past L1,
  // which may hold lines of an earlier batch's plan). Rows without an adapter
  // may so be written while A x still runs, which reads x and the plan only.
  volatile int* abort = &s_abort;
  const uint64_t lim = p.wait_limit_ns;
  // In place, the rows without an adapter are as they should be.
  const LoraShares shares((unsigned)__ldcg(p.meta + (p.base == p.out ? 0 : 1)) * (unsigned)p.g.NB, gridDim.x);
  const unsigned v0 = shares.begin(blockIdx.x), v1 = shares.begin(blockIdx.x + 1);
  // The tiles without an adapter are the last: only the epilogue sees them.
  const unsigned va = min(v1, (unsigned)__ldcg(p.meta) * (unsigned)p.g.NB);
  bool ok = true;
  // The first tile's u, which everything waits for, by the u and the epilogue
  // warps together, once the A x kernel has ended.
  auto first_u = [&](const LoraTile& t, int tile) {
    const LoraPieces pc = lora_pieces(p, shrink_shares(p), tile, t);
    pdl_wait();
    lora_u_operand<ACT, 2>(t, pc, p.g.max_r16, smem, warp - LB_WARP_U, LB_FIRST_WARPS, lane);
    fence_async_smem();
    named_bar_sync(1, LB_FIRST_WARPS * 32);
  };

  if (warp == 0) {
    RingPos rp;
    int issued = 0;
    for (unsigned v = v0; v < va && ok;) {
      const LoraSpan sp(v, va, p.g.NB);
      const LoraTile t = lora_tile(p, sp.tile);
      v += sp.n;
      const uint32_t bytes = (uint32_t)t.r16 * 128;
      const uint8_t* b = t.block + p.g.b_off + (size_t)sp.first * bytes;
      for (int i = 0; i < sp.n; ++i, b += bytes) {
        if (!__all_sync(0xffffffffu, mbar_wait(&empty[rp.slot], rp.ph ^ 1u, abort, lim))) {
          ok = false;
          break;
        }
        mbar_expect_tx_elect(&full[rp.slot], bytes);
        bulk_g2s_if(lane == 0, ring + rp.slot * stage_bytes, b, bytes, &full[rp.slot]);
        ++issued;
        rp.next(stages);
      }
    }
    if (!ok) {
      if (lane == 0) {
        s_abort = 1;
        set_status(p.status, DEV_TIMEOUT);
      }
      volatile int never = 0;
      for (int i = 0; i < stages && i < issued; ++i) {
        rp.back(stages);
        mbar_wait(&full[rp.slot], rp.ph, &never, lim);
      }
    }
  } else if (warp == 1) {
    RingPos rp;
    int ju = 0, unit = 0;
    const uint32_t idesc = idesc_kf16<ACT>(128, 64);
    for (unsigned v = v0; v < va && ok; ++ju) {
      const LoraSpan sp(v, va, p.g.NB);
      const LoraTile t = lora_tile(p, sp.tile);
      v += sp.n;
      const int ub = ju % u_bufs;
      ok = __all_sync(0xffffffffu, mbar_wait(&u_full[ub], (uint32_t)(ju / u_bufs) & 1u, abort, lim));
      const uint32_t hi = smem_u32(smem + ub * u_bytes), lo = hi + (uint32_t)LORA_TILE_ROWS * t.r16 * 2;
      for (int i = 0; i < sp.n && ok; ++i, ++unit) {
        const int buf = unit % LB_ACC;
        ok = __all_sync(0xffffffffu, mbar_wait(&acc_empty[buf], ((uint32_t)(unit / LB_ACC) & 1u) ^ 1u, abort, lim)) &&
             __all_sync(0xffffffffu, mbar_wait(&full[rp.slot], rp.ph, abort, lim));
        if (!ok) break;
        tc_fence_after();
        const uint32_t b = smem_u32(ring + rp.slot * stage_bytes), d = tmem + (uint32_t)buf * 64;
        for (int ks = 0; ks < t.r16 / 16; ++ks) {
          const uint64_t bd = smem_desc_plain(b + ks * 2 * 1024, 1024);
          const uint32_t off = (uint32_t)ks * 2 * LORA_TILE_ROWS * 16;
          umma_kf16_warp(d, smem_desc_plain(hi + off, LORA_TILE_ROWS * 16), bd, idesc, ks ? 1u : 0u);
          umma_kf16_warp(d, smem_desc_plain(lo + off, LORA_TILE_ROWS * 16), bd, idesc, 1u);
        }
        umma_commit_warp(&acc_full[buf]);
        umma_commit_warp(&empty[rp.slot]);
        rp.next(stages);
      }
      if (ok) umma_commit_warp(&u_empty[ub]);
    }
    if (!ok && lane == 0) {
      s_abort = 1;
      set_status(p.status, DEV_TIMEOUT);
    }
    umma_commit_warp(&mma_done);
    volatile int never = 0;
    mbar_wait(&mma_done, 0, &never, lim);
  } else if (warp < LB_WARP_EPI) {
    const LoraShares ks = shrink_shares(p);
    int ju = 0;
    for (unsigned v = v0; v < va; ++ju) {
      const LoraSpan sp(v, va, p.g.NB);
      const LoraTile t = lora_tile(p, sp.tile);
      v += sp.n;
      const int ub = ju % u_bufs;
      if (ju == 0) {
        first_u(t, sp.tile);
        pdl_trigger();
      } else {
        if (!__all_sync(0xffffffffu, mbar_wait(&u_empty[ub], ((uint32_t)(ju / u_bufs) & 1u) ^ 1u, abort, lim))) {
          if (lane == 0) {
            s_abort = 1;
            set_status(p.status, DEV_TIMEOUT);
          }
          break;
        }
        lora_u_operand<ACT, 4>(t, lora_pieces(p, ks, sp.tile, t), p.g.max_r16, smem + ub * u_bytes, warp - LB_WARP_U,
                            LB_U_WARPS, lane);
        fence_async_smem();
        __syncwarp();
      }
      if (lane == 0) mbar_arrive(&u_full[ub]);
    }
    if (ju == 0) {
      pdl_wait();
      pdl_trigger();
    }
  } else {
    const int e = warp - LB_WARP_EPI;
    const int group = e / LB_EPI_WARPS, quarter = warp & 3, half = (e >> 2) & 1;
    const int c = half * 32 + (lane & 3) * 8;  // the lane's 8 columns of a unit
    int unit = 0;
    for (unsigned v = v0; v < v1 && ok;) {
      const LoraSpan sp(v, v1, p.g.NB);
      const LoraTile t = lora_tile(p, sp.tile);
      const bool with = t.adapter >= 0;
      const float scale = with ? __ldcg(reinterpret_cast<const float*>(p.packed + p.g.scale_off) + t.adapter) : 0.0f;
      // The lane's rows: quarter * 32 + lane / 4 + 8 k; -1 past the tile's.
      int row[4];
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const int r = quarter * 32 + (lane >> 2) + 8 * k;
        row[k] = r < t.n ? __ldcg(p.perm + t.pos + r) : -1;
      }
      auto load = [&](int i, uint4* y) {  // the base values of unit i
        const int n = (sp.first + i) * 64 + c;
#pragma unroll
        for (int k = 0; k < 4; ++k)
          y[k] = p.base && row[k] >= 0 && i < sp.n && n < p.g.N
                     ? __ldcs(reinterpret_cast<const uint4*>(p.base + (size_t)row[k] * p.ldbase + n))
                     : make_uint4(0, 0, 0, 0);
      };
      float scales[ROW_POWERS<ACT> ? 4 : 1] = {scale};  // of the lane's rows
      // Unit i from its base values in y, which are then unit i + 4's.
      auto unit_of = [&](int i, uint4* y) {
        if (with) {
          const int buf = (unit + i) % LB_ACC;
          ok = __all_sync(0xffffffffu, mbar_wait(&acc_full[buf], (uint32_t)((unit + i) / LB_ACC) & 1u, abort, lim));
          if (!ok) return;
          tc_fence_after();
          const uint32_t at = tmem + ((uint32_t)(quarter * 32) << 16) + (uint32_t)buf * 64 + half * 32;
#pragma unroll
          for (int h = 0; h < 2; ++h) {  // 16 rows
            uint32_t w[16];
            tmem_ld16x256x4(at + ((uint32_t)(16 * h) << 16), w);
            tmem_wait_ld();
#pragma unroll
            for (int k = 0; k < 2; ++k) {
              uint32_t* yw = reinterpret_cast<uint32_t*>(&y[2 * h + k]);
#pragma unroll
              for (int j = 0; j < 4; ++j) {
                const float2 f = fma_x2(__uint_as_float(w[4 * j + 2 * k]), __uint_as_float(w[4 * j + 2 * k + 1]),
                                        scales[ROW_POWERS<ACT> ? 2 * h + k : 0], act_x2_to_f32<ACT>(yw[j]));
                yw[j] = f32_to_act_x2<ACT>(f.x, f.y);
              }
            }
          }
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(&acc_empty[buf]);
        }
        const int n = (sp.first + i) * 64 + c;
        if (n < p.g.N) {
#pragma unroll
          for (int k = 0; k < 4; ++k)
            if (row[k] >= 0) __stcs(reinterpret_cast<uint4*>(p.out + (size_t)row[k] * p.ldout + n), y[k]);
        }
        load(i + 4, y);
      };
      // Two sets of base values in flight, each in registers of its own (a copy
      // from one to the other would wait for the load).
      const int i0 = (unit & 1) != group;
      uint4 y0[4], y1[4];
      load(i0, y0);
      load(i0 + 2, y1);
      if (v == v0 && with) first_u(t, sp.tile);
      if constexpr (ROW_POWERS<ACT>) {  // after the A x kernel's end, which first_u waits for
        uint32_t bound[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const int r = quarter * 32 + (lane >> 2) + 8 * k;
          bound[k] = with && r < t.n ? __ldcg(p.bound + t.pos + r) : 0u;
        }
#pragma unroll
        for (int k = 0; k < 4; ++k) scales[k] = row_scale(scale, bound[k]);
      }
      for (int i = i0; i < sp.n && ok; i += 4) {
        unit_of(i, y0);
        if (i + 2 < sp.n && ok) unit_of(i + 2, y1);
      }
      unit += sp.n;
      v += sp.n;
    }
    if (!ok && lane == 0) {
      s_abort = 1;
      set_status(p.status, DEV_TIMEOUT);
    }
  }
  __syncwarp();
  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, LB_ACC * 64);
  }
}

static cudaError_t launch_plan(LoraParams& p, int tile_rows, cudaStream_t st) {
  static std::atomic<unsigned long long> done{0};
  p.tile_rows = tile_rows;
  cudaError_t e = ensure_smem_attr(lora_plan_kernel, lp_smem(LORA_MAX_SLOTS), done);
  if (e == cudaSuccess)
    e = launch_pdl(lora_plan_kernel, dim3(1), dim3(LP_THREADS), (size_t)lp_smem(p.g.slots), st, p);
  count_launches(1);
  return e;
}

template <int ACT>
static cudaError_t tiled_of(LoraParams p, int num_sms, cudaStream_t st) {
  static std::atomic<unsigned long long> done_a{0}, done_b{0};
  const int sa = la_smem(p.g.max_r16), sb = lb_smem(p.g.max_r16);
  const dim3 grid((unsigned)(num_sms < LORA_MAX_CTAS ? num_sms : LORA_MAX_CTAS));
  cudaError_t e = ensure_smem_attr(lora_shrink_kernel<ACT>, LT_SMEM + 1024, done_a);
  if (e == cudaSuccess) e = ensure_smem_attr(lora_expand_kernel<ACT>, LT_SMEM + 1024, done_b);
  if (e == cudaSuccess) e = launch_plan(p, LORA_TILE_ROWS, st);
  if (e == cudaSuccess) e = launch_pdl(lora_shrink_kernel<ACT>, grid, dim3(LA_THREADS), (size_t)sa, st, p);
  if (e == cudaSuccess) e = launch_pdl(lora_expand_kernel<ACT>, grid, dim3(LB_THREADS), (size_t)sb, st, p);
  count_launches(2);
  return e;
}

template <int ACT>
static cudaError_t forward_of(LoraParams p, int num_sms, cudaStream_t st) {
  if (p.T <= LS_MAX_T) return small_of<ACT, false>(p, st);
  if (lora_planned_small(p.g, p.T, num_sms)) {
    p.bound = nullptr;  // the small kernel's rows have theirs in shared memory
    const cudaError_t e = p.T <= LS_COUNT_T ? cudaSuccess : launch_plan(p, LS_TOK, st);
    return e == cudaSuccess ? small_of<ACT, true>(p, st) : e;
  }
  return tiled_of<ACT>(p, num_sms, st);
}

cudaError_t launch_lora_forward(const LoraParams& p, int num_sms, cudaStream_t st) {
  if (p.T == 0) return cudaSuccess;
  return p.act_type == ACT_F16 ? forward_of<ACT_F16>(p, num_sms, st) : forward_of<ACT_BF16>(p, num_sms, st);
}

}  // namespace hmoe
