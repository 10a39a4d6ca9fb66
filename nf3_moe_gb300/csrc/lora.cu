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
  return p.act_type == ACT_F16 ? forward_as<ACT_F16>(p, st) : forward_as<ACT_BF16>(p, st);
}

}  // namespace hmoe
