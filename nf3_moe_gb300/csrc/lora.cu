// lora.cu -- low-rank adapters of many requests beside a shared projection:
//   out[t] = base[t] + scale_a * B_a (A_a x[t]),  a = ids[t] (-1: none).
#include "common.cuh"
#include "internal.h"

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
    const int o = i / r16 * ur + i % r16;
    split_act<ACT>(v, u_hi + o, u_lo + o);
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

// ------------------------------------------------------------ larger batches
// u[t][r] = sum_k A[r][k] x[t][k]: one warp per row and rank.
template <int ACT>
__global__ void lora_shrink_kernel(LoraParams p) {
  pdl_wait();
  pdl_trigger();
  const int lane = threadIdx.x & 31;
  const long long w = blockIdx.x * (long long)(blockDim.x >> 5) + (threadIdx.x >> 5);
  const int t = (int)(w / p.g.max_r16), r = (int)(w % p.g.max_r16);
  if (t >= p.T) return;
  const int a = lora_slot(p, t);
  if (a < 0) return;
  const int rank = reinterpret_cast<const int*>(p.packed)[a];
  if (r >= rank) return;
  const int r16 = (rank + 15) / 16 * 16;
  const uint8_t* block = p.packed + p.g.block_off + (size_t)a * p.g.block_bytes;
  const uint16_t* x = p.x + (size_t)t * p.ldx;
  float acc = 0.0f;
  for (int k = lane; k < p.g.K; k += 32)
    acc = fmaf(act_f32<ACT>(*reinterpret_cast<const uint16_t*>(block + lora_a_byte(r16, r, k))), act_f32<ACT>(x[k]), acc);
#pragma unroll
  for (int d = 16; d > 0; d >>= 1) acc += __shfl_xor_sync(0xffffffffu, acc, d);
  if (lane == 0) p.u[(size_t)t * p.g.max_r16 + r] = acc;
}

// out[t][n] = base[t][n] + scale * sum_r B[n][r] u[t][r]: one thread per output.
template <int ACT>
__global__ void lora_expand_kernel(LoraParams p) {
  pdl_wait();
  pdl_trigger();
  const int t = blockIdx.x;
  const int n = blockIdx.y * blockDim.x + threadIdx.x;
  if (n >= p.g.N) return;
  const int a = lora_slot(p, t);
  float acc = 0.0f;
  if (a >= 0) {
    const int rank = reinterpret_cast<const int*>(p.packed)[a];
    const float scale = reinterpret_cast<const float*>(p.packed + p.g.scale_off)[a];
    const int r16 = (rank + 15) / 16 * 16;
    const uint8_t* b = p.packed + p.g.block_off + (size_t)a * p.g.block_bytes + p.g.b_off;
    const float* u = p.u + (size_t)t * p.g.max_r16;
    for (int r = 0; r < rank; ++r)
      acc = fmaf(act_f32<ACT>(*reinterpret_cast<const uint16_t*>(b + lora_b_byte(r16, n, r))), u[r], acc);
    acc *= scale;
  }
  const float y = p.base ? act_f32<ACT>(p.base[(size_t)t * p.ldbase + n]) : 0.0f;
  p.out[(size_t)t * p.ldout + n] = f32_to_act<ACT>(y + acc);
}

template <int ACT>
static cudaError_t forward_as(const LoraParams& p, cudaStream_t st) {
  const long long warps = (long long)p.T * p.g.max_r16;
  cudaError_t e = launch_pdl(lora_shrink_kernel<ACT>, dim3((unsigned)((warps + 7) / 8)), dim3(256), 0, st, p);
  if (e == cudaSuccess)
    e = launch_pdl(lora_expand_kernel<ACT>, dim3((unsigned)p.T, (unsigned)((p.g.N + 255) / 256)), dim3(256), 0, st, p);
  count_launches(2);
  return e;
}

cudaError_t launch_lora_forward(const LoraParams& p, int num_sms, cudaStream_t st) {
  if (p.T == 0) return cudaSuccess;
  if (p.T <= LS_MAX_T) return p.act_type == ACT_F16 ? small_of<ACT_F16>(p, st) : small_of<ACT_BF16>(p, st);
  return p.act_type == ACT_F16 ? forward_as<ACT_F16>(p, st) : forward_as<ACT_BF16>(p, st);
}

}  // namespace hmoe
