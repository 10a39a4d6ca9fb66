// lora.cu -- low-rank adapters of many requests beside a shared projection:
//   out[t] = base[t] + scale_a * B_a (A_a x[t]),  a = ids[t] (-1: none).
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
// Byte of B[n][r] from the start of the block's B tiles.
__host__ __device__ __forceinline__ size_t lora_b_byte(int r16, int n, int r) {
  return (size_t)(n >> 6) * r16 * 128 + ((size_t)(r >> 3) * 64 + (n & 63)) * 16 + (r & 7) * 2;
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
// A cluster of LS_C CTAs serves up to LS_TOK rows of one adapter: CTA c sums
// A x over its share of K, the CTAs exchange their partial sums through
// distributed shared memory, and each adds B u for its share of N. The batch
// is grouped without a pass of its own: cluster t belongs to row t, and goes
// on only if row t is the first of a group, that is if the number of earlier
// rows with the same id is a multiple of LS_TOK.
//
// Both products run on mma.sync m16n8k16 with the rows on the M side and the
// weights, straight from global memory, on the N side. K inside a group of 32
// (and the rank in the second product) is permuted alike for both operands, so
// that a lane's operand words are 16 bytes of one row. The columns of the
// second product are permuted so that a lane ends up with 8 neighbouring ones.
constexpr int LS_C = 8;
constexpr int LS_THREADS = 256;
constexpr int LS_WARPS = LS_THREADS / 32;
constexpr int LS_TOK = 16;
constexpr int LS_MAX_T = LS_THREADS;  // the grouping looks at one row a thread

__device__ __forceinline__ uint32_t ls_cluster_rank() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}
__device__ __forceinline__ float ld_cluster_f32(const void* p, uint32_t rank) {
  uint32_t a;
  float v;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"(smem_u32(p)), "r"(rank));
  asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(a) : "memory");
  return v;
}
__device__ __forceinline__ void cluster_arrive() { asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory"); }
__device__ __forceinline__ void cluster_wait() { asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory"); }
__device__ __forceinline__ uint4 ldg16(const void* p) { return __ldg(static_cast<const uint4*>(p)); }

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

// R: the largest padded rank of the set, rounded up to 16, 32, 64 or 128.
template <int ACT, int R>
__global__ void __cluster_dims__(LS_C, 1, 1) __launch_bounds__(LS_THREADS) lora_small_kernel(LoraParams p) {
  extern __shared__ __align__(16) uint8_t ls_sm[];
  __shared__ int s_tok[LS_TOK], s_cnt[LS_WARPS];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int cta = (int)ls_cluster_rank();
  const int t0 = blockIdx.y;
  pdl_wait();
  pdl_trigger();
  const int a = lora_slot(p, t0);
  const int rank = a >= 0 ? reinterpret_cast<const int*>(p.packed)[a] : 0;
  const int n0 = cta * p.g.NB / LS_C * 64, n1 = min(p.g.N, (cta + 1) * p.g.NB / LS_C * 64);
  if (rank == 0) {  // base alone
    if (p.base != p.out)
      for (int n = n0 + tid * 8; n < n1; n += LS_THREADS * 8)
        *reinterpret_cast<uint4*>(p.out + (size_t)t0 * p.ldout + n) =
            p.base ? *reinterpret_cast<const uint4*>(p.base + (size_t)t0 * p.ldbase + n) : make_uint4(0, 0, 0, 0);
    return;
  }
  // The group: T <= LS_THREADS, so thread j looks at row j.
  const bool same = tid < p.T && p.ids[tid] == a;
  if (__syncthreads_count(same && tid < t0) % LS_TOK != 0) return;
  const unsigned later = __ballot_sync(0xffffffffu, same && tid >= t0);
  if (lane == 0) s_cnt[warp] = __popc(later);
  if (tid < LS_TOK) s_tok[tid] = -1;
  __syncthreads();
  {
    int pos = __popc(later & ((1u << lane) - 1u));
    for (int w = 0; w < warp; ++w) pos += s_cnt[w];
    if (same && tid >= t0 && pos < LS_TOK) s_tok[pos] = tid;
  }
  __syncthreads();
  const float scale = reinterpret_cast<const float*>(p.packed + p.g.scale_off)[a];
  const int r16 = (rank + 15) / 16 * 16;
  const uint8_t* block = p.packed + p.g.block_off + (size_t)a * p.g.block_bytes;
  const uint8_t* btiles = block + p.g.b_off;
  const int g = lane >> 2, q = lane & 3;
  const int ta = s_tok[g], tb = s_tok[g + 8];

  // ---- A x over this CTA's k-blocks, half a block (32 of K) a step
  float acc[R / 8][4];
#pragma unroll
  for (int j = 0; j < R / 8; ++j)
#pragma unroll
    for (int i = 0; i < 4; ++i) acc[j][i] = 0.0f;
  const int h0 = 2 * (cta * p.g.KB / LS_C), h1 = 2 * ((cta + 1) * p.g.KB / LS_C);
  for (int h = h0 + warp; h < h1; h += LS_WARPS) {
    const int k = h * 32 + q * 8;
    const uint4 zero = make_uint4(0, 0, 0, 0);
    const uint4 xa = (ta >= 0 && k < p.g.K) ? ldg16(p.x + (size_t)ta * p.ldx + k) : zero;
    const uint4 xb = (tb >= 0 && k < p.g.K) ? ldg16(p.x + (size_t)tb * p.ldx + k) : zero;
    const uint8_t* tile = block + (size_t)(h >> 1) * r16 * 128 + g * 128 + ((((h & 1) * 4 + q) ^ g) * 16);
#pragma unroll
    for (int j = 0; j < R / 8; ++j) {
      if (8 * j < r16) {
        const uint4 w = ldg16(tile + j * 1024);
        mma_16816<ACT>(acc[j], xa.x, xb.x, xa.y, xb.y, w.x, w.y);
        mma_16816<ACT>(acc[j], xa.z, xb.z, xa.w, xb.w, w.z, w.w);
      }
    }
  }
  float* part = reinterpret_cast<float*>(ls_sm);
  float* sum = part + LS_WARPS * LS_TOK * r16;
  uint16_t* u_hi = reinterpret_cast<uint16_t*>(sum + LS_TOK * r16);
  const int ur = r16 + 8;  // row stride of u: 16-byte rows in different banks
  uint16_t* u_lo = u_hi + LS_TOK * ur;
#pragma unroll
  for (int j = 0; j < R / 8; ++j) {
    if (8 * j < r16) {
      float* d = part + (warp * LS_TOK + g) * r16 + 8 * j + 2 * q;
      *reinterpret_cast<float2*>(d) = make_float2(acc[j][0], acc[j][1]);
      *reinterpret_cast<float2*>(d + 8 * r16) = make_float2(acc[j][2], acc[j][3]);
    }
  }
  __syncthreads();
  for (int i = tid; i < LS_TOK * r16; i += LS_THREADS) {
    float v = 0.0f;
#pragma unroll
    for (int w = 0; w < LS_WARPS; ++w) v += part[w * LS_TOK * r16 + i];
    sum[i] = v;
  }
  cluster_arrive();
  cluster_wait();
  for (int i = tid; i < LS_TOK * r16; i += LS_THREADS) {
    float v = 0.0f;
#pragma unroll
    for (int c = 0; c < LS_C; ++c) v += ld_cluster_f32(sum + i, c);  // the same order in every CTA
    const int row = i / r16, r = i - row * r16;
    // past the rank A's zeros met whatever x held
    split_act<ACT>(r < rank ? v : 0.0f, u_hi + row * ur + r, u_lo + row * ur + r);
  }
  __syncthreads();
  cluster_arrive();  // this CTA has read the others' sums

  // ---- B u over this CTA's columns, 32 a step
  for (int n = n0 + warp * 32; n < n1; n += LS_WARPS * 32) {
    float d[4][4];
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int e = 0; e < 4; ++e) d[i][e] = 0.0f;
    // column c of MMA i is n + 8 (c / 2) + 2 i + c % 2
    const uint8_t* tile = btiles + (size_t)(n >> 6) * r16 * 128 + ((n & 63) + 8 * (g >> 1) + (g & 1)) * 16;
#pragma unroll
    for (int r = 0; r < R; r += 16) {
      if (r < r16) {
        // ranks r + 4 q .. r + 4 q + 3 of this lane
        const uint2 ha = *reinterpret_cast<const uint2*>(u_hi + g * ur + r + 4 * q);
        const uint2 hb = *reinterpret_cast<const uint2*>(u_hi + (g + 8) * ur + r + 4 * q);
        const uint2 la = *reinterpret_cast<const uint2*>(u_lo + g * ur + r + 4 * q);
        const uint2 lb = *reinterpret_cast<const uint2*>(u_lo + (g + 8) * ur + r + 4 * q);
        const uint8_t* src = tile + (r / 8 + (q >> 1)) * 1024 + (q & 1) * 8;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const uint2 w = __ldg(reinterpret_cast<const uint2*>(src + i * 32));
          mma_16816<ACT>(d[i], ha.x, hb.x, ha.y, hb.y, w.x, w.y);
          mma_16816<ACT>(d[i], la.x, lb.x, la.y, lb.y, w.x, w.y);
        }
      }
    }
    const int c = n + 8 * q;
    if (c < p.g.N) {
#pragma unroll
      for (int half = 0; half < 2; ++half) {
        const int t = half ? tb : ta;
        if (t < 0) continue;
        uint4 y = p.base ? *reinterpret_cast<const uint4*>(p.base + (size_t)t * p.ldbase + c)
                         : make_uint4(0, 0, 0, 0);
        uint32_t* yw = reinterpret_cast<uint32_t*>(&y);
#pragma unroll
        for (int i = 0; i < 4; ++i)
          yw[i] = f32x2_to_act<ACT>(fmaf(scale, d[i][2 * half], act_f32<ACT>((uint16_t)(yw[i] & 0xFFFFu))),
                                    fmaf(scale, d[i][2 * half + 1], act_f32<ACT>((uint16_t)(yw[i] >> 16))));
        *reinterpret_cast<uint4*>(p.out + (size_t)t * p.ldout + c) = y;
      }
    }
  }
  cluster_wait();  // the others have read this CTA's sums
}

template <int ACT, int R>
static cudaError_t small_as(const LoraParams& p, cudaStream_t st) {
  static std::atomic<unsigned long long> done{0};
  const int smem = ls_smem(p.g.max_r16);
  cudaError_t e = ensure_smem_attr(lora_small_kernel<ACT, R>, ls_smem(R), done);
  if (e == cudaSuccess)
    e = launch_pdl(lora_small_kernel<ACT, R>, dim3(LS_C, (unsigned)p.T), dim3(LS_THREADS), (size_t)smem, st, p);
  count_launches(1);
  return e;
}
template <int ACT>
static cudaError_t small_of(const LoraParams& p, cudaStream_t st) {
  if (p.g.max_r16 <= 16) return small_as<ACT, 16>(p, st);
  if (p.g.max_r16 <= 32) return small_as<ACT, 32>(p, st);
  if (p.g.max_r16 <= 64) return small_as<ACT, 64>(p, st);
  return small_as<ACT, 128>(p, st);
}

// ------------------------------------------------------------ larger batches: plan, A x, B u
// Three launches. The plan groups the rows by adapter and cuts the groups into
// tiles of up to 128 rows; the rows of a tile sit on the M side of tcgen05.mma
// and the adapter on its N side.

// One CTA. Rows without an adapter (or with an empty slot) form the last group.
// The order of the rows inside a group does not matter to any result.
constexpr int LP_THREADS = 1024;
__global__ void __launch_bounds__(LP_THREADS) lora_plan_kernel(LoraParams p) {
  __shared__ int s_cnt[LORA_MAX_SLOTS + 1], s_rank[LORA_MAX_SLOTS + 1], s_wsum[2][LP_THREADS / 32];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int G = p.g.slots + 1;
  for (int g = tid; g < G; g += LP_THREADS) s_cnt[g] = 0;
  pdl_wait();
  pdl_trigger();
  for (int g = tid; g < G; g += LP_THREADS) s_rank[g] = g < p.g.slots ? reinterpret_cast<const int*>(p.packed)[g] : 0;
  __syncthreads();
  auto group_of = [&](int t) {
    const int a = lora_slot(p, t);
    return a >= 0 && s_rank[a] > 0 ? a : G - 1;
  };
  // The place of a row in its group, one atomic per group and warp; kept in
  // the u scratch, which nothing else uses yet.
  int* place = reinterpret_cast<int*>(p.u);
  for (int t0 = warp * 32; t0 < p.T; t0 += LP_THREADS) {
    const int t = t0 + lane;
    const int g = t < p.T ? group_of(t) : -1;
    const unsigned peers = __match_any_sync(0xffffffffu, g);
    const int first = __ffs(peers) - 1;
    int base = 0;
    if (lane == first && g >= 0) base = atomicAdd(&s_cnt[g], __popc(peers));
    base = __shfl_sync(0xffffffffu, base, first);
    if (g >= 0) place[t] = base + __popc(peers & ((1u << lane) - 1u));
  }
  __syncthreads();
  // Exclusive scans of the groups' rows and tiles (G <= 513 <= LP_THREADS).
  const int n = tid < G ? s_cnt[tid] : 0, nt = (n + LORA_TILE_ROWS - 1) / LORA_TILE_ROWS;
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
  int bn = 0, bt = 0;
  for (int w = 0; w < warp; ++w) {
    bn += s_wsum[0][w];
    bt += s_wsum[1][w];
  }
  const int row0 = bn + in - n, tile0 = bt + it - nt;
  __syncthreads();
  if (tid < G) {
    s_cnt[tid] = row0;  // from here on: where the group starts
    for (int j = 0; j < nt; ++j) {
      p.tiles[tile0 + j] = make_int4(tid < G - 1 ? tid : -1, row0 + j * LORA_TILE_ROWS,
                                     min(LORA_TILE_ROWS, n - j * LORA_TILE_ROWS), 0);
      p.arrived[tile0 + j] = 0;
    }
    if (tid == G - 1) {
      const int with = tile0;
      p.meta[0] = with;
      p.meta[1] = tile0 + nt;
      p.meta[3] = row0;
      const int s = with > 0 ? (LORA_SPLIT_ITEMS + with - 1) / with : 1;
      p.meta[2] = max(1, min(min(s, LORA_MAX_SPLITS), p.g.KB));
    }
  }
  __syncthreads();
  for (int t = tid; t < p.T; t += LP_THREADS) p.perm[s_cnt[group_of(t)] + place[t]] = t;
}

__device__ __forceinline__ void cp_async16(void* dst, const void* src, uint32_t bytes) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(smem_u32(dst)), "l"(src), "r"(bytes) : "memory");
}
__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_async_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

constexpr int LT_THREADS = 256;
constexpr int LT_STAGES = 4;
constexpr int LT_X_BYTES = LORA_TILE_ROWS * 128;  // 128 rows x 64 values

// Shared memory of the A x kernel: the stages' x tiles and A tiles.
__host__ __device__ constexpr int lt_shrink_smem(int r16) { return 1024 + LT_STAGES * (LT_X_BYTES + r16 * 128); }

// u[split][pos][r] = A x over one K split of one tile; the last split of a
// tile to finish adds the others' sums to split 0, in order.
template <int ACT>
__global__ void __launch_bounds__(LT_THREADS) lora_shrink_kernel(LoraParams p) {
  extern __shared__ uint8_t lt_sm[];
  __shared__ __align__(8) uint64_t s_free[LT_STAGES];
  __shared__ uint32_t s_tmem;
  __shared__ int s_tok[LORA_TILE_ROWS], s_abort, s_last;
  uint8_t* smem = lt_sm + ((1024u - (smem_u32(lt_sm) & 1023u)) & 1023u);
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const uint32_t cols = p.g.max_r16 <= 32 ? 32u : (p.g.max_r16 <= 64 ? 64u : 128u);
  if (warp == 0) {
    tmem_alloc(&s_tmem, cols);
    tmem_relinquish();
  }
  if (tid == 0) {
    for (int i = 0; i < LT_STAGES; ++i) mbar_init(&s_free[i], 1);
    fence_mbar_init();
    s_abort = 0;
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = s_tmem;
  pdl_wait();
  pdl_trigger();  // after the TMEM allocation: the next kernel's may then wait for this one's end
  const int splits = p.meta[2];
  const int items = p.meta[0] * splits;
  const size_t split_rows = (size_t)p.meta[3];
  uint32_t phase = 0;  // bit i: parity of stage i's next completion
  bool ok = true;
  for (int item = blockIdx.x; item < items && ok; item += gridDim.x) {
    const int tile = item / splits, split = item - tile * splits;
    const int4 ti = p.tiles[tile];
    const int rank = reinterpret_cast<const int*>(p.packed)[ti.x];
    const int r16 = (rank + 15) / 16 * 16;
    const uint8_t* A = p.packed + p.g.block_off + (size_t)ti.x * p.g.block_bytes;
    const int kb0 = (int)((long long)split * p.g.KB / splits), nk = (int)((long long)(split + 1) * p.g.KB / splits) - kb0;
    if (tid < LORA_TILE_ROWS) s_tok[tid] = tid < ti.z ? p.perm[ti.y + tid] : -1;
    __syncthreads();
    // This thread's copies: chunk c of rows tid / 8 + 32 i.
    const int c = tid & 7;
    const uint16_t* src[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int t = s_tok[(tid >> 3) + 32 * i];
      src[i] = t < 0 ? nullptr : p.x + (size_t)t * p.ldx;
    }
    const int stage_bytes = LT_X_BYTES + r16 * 128;
    auto load = [&](int i) {
      uint8_t* st = smem + (i % LT_STAGES) * stage_bytes;
      const int k = (kb0 + i) * 64 + c * 8;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int r = (tid >> 3) + 32 * j;
        if (src[j]) cp_async16(st + r * 128 + ((c ^ (r & 7)) * 16), src[j] + (k < p.g.K ? k : 0), k < p.g.K ? 16u : 0u);
      }
      const uint8_t* a = A + (size_t)(kb0 + i) * r16 * 128;
      for (int j = tid; j < r16 * 8; j += LT_THREADS) cp_async16(st + LT_X_BYTES + j * 16, a + j * 16, 16u);
    };
#pragma unroll
    for (int i = 0; i < LT_STAGES - 1; ++i) {
      if (i < nk) load(i);
      cp_async_commit();
    }
    const uint32_t idesc = idesc_kf16<ACT>(128, r16);
    for (int i = 0; i < nk; ++i) {
      cp_async_wait<LT_STAGES - 2>();
      fence_async_smem();
      if (__syncthreads_or(!ok)) {
        ok = false;
        break;
      }
      const int s = i % LT_STAGES;
      if (warp == 0) {
        const uint32_t x_lo = smem_desc_sw128_lo(smem_u32(smem + s * stage_bytes));
        const uint32_t a_lo = smem_desc_sw128_lo(smem_u32(smem + s * stage_bytes + LT_X_BYTES));
#pragma unroll
        for (int ks = 0; ks < 4; ++ks)
          umma_kf16_warp(tmem, desc_from_lo(x_lo + 2 * ks), desc_from_lo(a_lo + 2 * ks), idesc, (i | ks) ? 1u : 0u);
        umma_commit_warp(&s_free[s]);
      }
      // Refill the stage that the previous k-block's MMAs read.
      if (i > 0) {
        const int f = (i - 1) % LT_STAGES;
        ok = mbar_wait(&s_free[f], (phase >> f) & 1u, &s_abort, p.wait_limit_ns) && ok;
        phase ^= 1u << f;
      }
      if (ok && i + LT_STAGES - 1 < nk) load(i + LT_STAGES - 1);
      cp_async_commit();
    }
    if (ok) {
      const int f = (nk - 1) % LT_STAGES;
      ok = mbar_wait(&s_free[f], (phase >> f) & 1u, &s_abort, p.wait_limit_ns);
      phase ^= 1u << f;
    }
    if (__syncthreads_or(!ok)) {
      ok = false;
      break;
    }
    tc_fence_after();
    // Lane = row. The two warps of a quarter take alternate 16 columns.
    const int row = (warp & 3) * 32 + lane;
    float* u = p.u + (split * split_rows + ti.y + row) * p.g.max_r16;
    for (int col = (warp >> 2) * 16; col < r16; col += 32) {
      uint32_t v[16];
      tmem_ld16(tmem + ((uint32_t)((warp & 3) * 32) << 16) + col, v);
      tmem_wait_ld();
      if (row < ti.z) {
#pragma unroll
        for (int j = 0; j < 4; ++j)
          *reinterpret_cast<uint4*>(u + col + 4 * j) = make_uint4(v[4 * j], v[4 * j + 1], v[4 * j + 2], v[4 * j + 3]);
      }
    }
    tc_fence_before();
    if (splits > 1) {
      __threadfence();
      __syncthreads();
      if (tid == 0) s_last = atomicAdd(&p.arrived[tile], 1) == splits - 1;
      __syncthreads();
      if (s_last) {
        __threadfence();
        const int per = r16 / 4;
        for (int j = tid; j < ti.z * per; j += LT_THREADS) {
          float* d = p.u + ((size_t)ti.y + j / per) * p.g.max_r16 + (j % per) * 4;
          float4 sum = __ldcg(reinterpret_cast<const float4*>(d));
          for (int q = 1; q < splits; ++q) {
            const float4 v = __ldcg(reinterpret_cast<const float4*>(d + q * split_rows * p.g.max_r16));
            sum.x += v.x;
            sum.y += v.y;
            sum.z += v.z;
            sum.w += v.w;
          }
          *reinterpret_cast<float4*>(d) = sum;
        }
      }
    }
    __syncthreads();
    tc_fence_after();
  }
  if (!ok) {
    if (tid == 0) set_status(p.status, DEV_TIMEOUT);
    s_abort = 1;
  }
  cp_async_wait<0>();
  tc_fence_before();
  __syncthreads();
  if (warp == 0) {
    tc_fence_after();
    tmem_dealloc(tmem, cols);
  }
}

// Shared memory of the B u kernel: u's two parts and the stages' base tiles
// and B tiles.
constexpr int LX_STAGES = 3;
constexpr int LX_TILE_BYTES = LORA_TILE_ROWS * 128;  // 128 rows x 64 columns
__host__ __device__ constexpr int lx_smem(int r16) {
  return 1024 + 2 * LORA_TILE_ROWS * r16 * 2 + LX_STAGES * (LX_TILE_BYTES + r16 * 128);
}

// out = base + scale B u. The (tile, 64 columns) units of the batch, tiles
// slowest, are dealt to the CTAs in contiguous shares.
template <int ACT>
__global__ void __launch_bounds__(LT_THREADS) lora_expand_kernel(LoraParams p) {
  extern __shared__ uint8_t lt_sm[];
  __shared__ __align__(8) uint64_t s_full[2];
  __shared__ uint32_t s_tmem;
  __shared__ int s_tok[LORA_TILE_ROWS], s_abort;
  uint8_t* smem = lt_sm + ((1024u - (smem_u32(lt_sm) & 1023u)) & 1023u);
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  if (warp == 0) {
    tmem_alloc(&s_tmem, 128);
    tmem_relinquish();
  }
  if (tid == 0) {
    mbar_init(&s_full[0], 1);
    mbar_init(&s_full[1], 1);
    fence_mbar_init();
    s_abort = 0;
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = s_tmem;
  pdl_wait();
  pdl_trigger();
  // In place, the rows without an adapter are as they should be.
  const long long units = (long long)(p.base == p.out ? p.meta[0] : p.meta[1]) * p.g.NB;
  long long v0 = units * blockIdx.x / gridDim.x;
  const long long v1 = units * (blockIdx.x + 1) / gridDim.x;
  uint32_t phase = 0;
  bool ok = true;
  while (v0 < v1 && ok) {
    const int tile = (int)(v0 / p.g.NB), nt0 = (int)(v0 % p.g.NB);
    const int nn = (int)min(v1 - v0, (long long)(p.g.NB - nt0));
    v0 += nn;
    const int4 ti = p.tiles[tile];
    const bool with = ti.x >= 0;
    const int rank = with ? reinterpret_cast<const int*>(p.packed)[ti.x] : 0;
    const float scale = with ? reinterpret_cast<const float*>(p.packed + p.g.scale_off)[ti.x] : 0.0f;
    const int r16 = (rank + 15) / 16 * 16;
    const uint8_t* B = p.packed + p.g.block_off + (size_t)(with ? ti.x : 0) * p.g.block_bytes + p.g.b_off;
    if (tid < LORA_TILE_ROWS) s_tok[tid] = tid < ti.z ? p.perm[ti.y + tid] : -1;
    __syncthreads();
    uint8_t* u_hi = smem;
    uint8_t* u_lo = smem + LORA_TILE_ROWS * r16 * 2;
    uint8_t* ring = u_lo + LORA_TILE_ROWS * r16 * 2;
    const int stage_bytes = LX_TILE_BYTES + r16 * 128;
    const int c = tid & 7;
    int tok[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) tok[j] = s_tok[(tid >> 3) + 32 * j];
    auto load = [&](int i) {
      uint8_t* st = ring + (i % LX_STAGES) * stage_bytes;
      const int n = (nt0 + i) * 64 + c * 8;
      if (p.base && n < p.g.N) {
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const int r = (tid >> 3) + 32 * j;
          if (tok[j] >= 0) cp_async16(st + r * 128 + ((c ^ (r & 7)) * 16), p.base + (size_t)tok[j] * p.ldbase + n, 16u);
        }
      }
      const uint8_t* b = B + (size_t)(nt0 + i) * r16 * 128;
      for (int j = tid; j < r16 * 8; j += LT_THREADS) cp_async16(st + LX_TILE_BYTES + j * 16, b + j * 16, 16u);
    };
#pragma unroll
    for (int i = 0; i < LX_STAGES - 1; ++i) {
      if (i < nn) load(i);
      cp_async_commit();
    }
    // u's two parts as the A operand: 16-byte core-matrix rows, [r16 / 8][128 rows].
    {
      const int row = tid & (LORA_TILE_ROWS - 1);
      const float* u = p.u + ((size_t)ti.y + row) * p.g.max_r16;
      for (int ch = tid >> 7; ch < r16 / 8; ch += LT_THREADS / LORA_TILE_ROWS) {
        uint16_t hi[8], lo[8];
        float f[8] = {0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f};
        if (row < ti.z) {
          *reinterpret_cast<float4*>(f) = __ldcg(reinterpret_cast<const float4*>(u + ch * 8));
          *reinterpret_cast<float4*>(f + 4) = __ldcg(reinterpret_cast<const float4*>(u + ch * 8 + 4));
        }
#pragma unroll
        for (int j = 0; j < 8; ++j) split_act<ACT>(ch * 8 + j < rank ? f[j] : 0.0f, &hi[j], &lo[j]);
        *reinterpret_cast<uint4*>(u_hi + (ch * LORA_TILE_ROWS + row) * 16) = *reinterpret_cast<const uint4*>(hi);
        *reinterpret_cast<uint4*>(u_lo + (ch * LORA_TILE_ROWS + row) * 16) = *reinterpret_cast<const uint4*>(lo);
      }
    }
    const uint32_t idesc = idesc_kf16<ACT>(128, 64);
    auto issue = [&](int i) {  // the MMAs of unit i, by a converged warp
      const uint32_t b = smem_u32(ring + (i % LX_STAGES) * stage_bytes + LX_TILE_BYTES);
      const uint32_t d = tmem + (uint32_t)(i & 1) * 64;
      for (int ks = 0; ks < r16 / 16; ++ks) {
        const uint64_t bd = smem_desc_plain(b + ks * 2 * 1024, 1024);
        const uint32_t off = (uint32_t)ks * 2 * LORA_TILE_ROWS * 16;
        umma_kf16_warp(d, smem_desc_plain(smem_u32(u_hi) + off, LORA_TILE_ROWS * 16), bd, idesc, ks ? 1u : 0u);
        umma_kf16_warp(d, smem_desc_plain(smem_u32(u_lo) + off, LORA_TILE_ROWS * 16), bd, idesc, 1u);
      }
      umma_commit_warp(&s_full[i & 1]);
    };
    // Before unit i's epilogue the MMAs of unit i + 1 are issued.
    for (int i = -1; i < nn; ++i) {
      if (i + 1 < nn) cp_async_wait<LX_STAGES - 2>();
      fence_async_smem();
      tc_fence_before();
      if (__syncthreads_or(!ok)) {
        ok = false;
        break;
      }
      tc_fence_after();
      if (with && i + 1 < nn && warp == 0) issue(i + 1);
      if (i < 0) {
        if (LX_STAGES - 1 < nn) load(LX_STAGES - 1);
        cp_async_commit();
        continue;
      }
      uint8_t* st = ring + (i % LX_STAGES) * stage_bytes;
      if (with) {
        ok = mbar_wait(&s_full[i & 1], (phase >> (i & 1)) & 1u, &s_abort, p.wait_limit_ns);
        phase ^= 1u << (i & 1);
        __syncwarp();
        tc_fence_after();
        const int row = (warp & 3) * 32 + lane, half = warp >> 2;
        uint32_t v[32];
        tmem_ld32(tmem + ((uint32_t)((warp & 3) * 32) << 16) + (uint32_t)(i & 1) * 64 + half * 32, v);
        tmem_wait_ld();
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          uint4* at = reinterpret_cast<uint4*>(st + row * 128 + (((half * 4 + j) ^ (row & 7)) * 16));
          uint4 y = p.base ? *at : make_uint4(0, 0, 0, 0);
          uint32_t* yw = reinterpret_cast<uint32_t*>(&y);
#pragma unroll
          for (int w = 0; w < 4; ++w)
            yw[w] = f32x2_to_act<ACT>(
                fmaf(scale, __uint_as_float(v[8 * j + 2 * w]), act_f32<ACT>((uint16_t)(yw[w] & 0xFFFFu))),
                fmaf(scale, __uint_as_float(v[8 * j + 2 * w + 1]), act_f32<ACT>((uint16_t)(yw[w] >> 16))));
          *at = y;
        }
        __syncthreads();
      }
      const int n = (nt0 + i) * 64 + c * 8;
      if (n < p.g.N) {
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const int r = (tid >> 3) + 32 * j;
          if (tok[j] >= 0)
            *reinterpret_cast<uint4*>(p.out + (size_t)tok[j] * p.ldout + n) =
                with || p.base ? *reinterpret_cast<const uint4*>(st + r * 128 + ((c ^ (r & 7)) * 16))
                               : make_uint4(0, 0, 0, 0);
        }
      }
      // A thread refills the chunks it has just stored; B's tile was read by MMAs that have completed.
      if (i + LX_STAGES < nn) load(i + LX_STAGES);
      cp_async_commit();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
  }
  if (!ok) {
    if (tid == 0) set_status(p.status, DEV_TIMEOUT);
    s_abort = 1;
  }
  cp_async_wait<0>();
  tc_fence_before();
  __syncthreads();
  if (warp == 0) {
    tc_fence_after();
    tmem_dealloc(tmem, 128);
  }
}

template <int ACT>
static cudaError_t tiled_as(const LoraParams& p, int num_sms, cudaStream_t st) {
  static std::atomic<unsigned long long> done_a{0}, done_b{0};
  const int sa = lt_shrink_smem(p.g.max_r16), sb = lx_smem(p.g.max_r16);
  cudaError_t e = ensure_smem_attr(lora_shrink_kernel<ACT>, lt_shrink_smem(LORA_MAX_RANK), done_a);
  if (e == cudaSuccess) e = ensure_smem_attr(lora_expand_kernel<ACT>, lx_smem(LORA_MAX_RANK), done_b);
  if (e == cudaSuccess) e = launch_pdl(lora_plan_kernel, dim3(1), dim3(LP_THREADS), 0, st, p);
  if (e == cudaSuccess) e = launch_pdl(lora_shrink_kernel<ACT>, dim3(2 * num_sms), dim3(LT_THREADS), (size_t)sa, st, p);
  if (e == cudaSuccess) e = launch_pdl(lora_expand_kernel<ACT>, dim3(2 * num_sms), dim3(LT_THREADS), (size_t)sb, st, p);
  count_launches(3);
  return e;
}

cudaError_t launch_lora_forward(const LoraParams& p, int num_sms, cudaStream_t st) {
  if (p.T == 0) return cudaSuccess;
  if (p.T <= LS_MAX_T) return p.act_type == ACT_F16 ? small_of<ACT_F16>(p, st) : small_of<ACT_BF16>(p, st);
  return p.act_type == ACT_F16 ? tiled_as<ACT_F16>(p, num_sms, st) : tiled_as<ACT_BF16>(p, num_sms, st);
}

}  // namespace hmoe
