// topk.cuh -- the order of logits that the routing and the few-token layer choose by, and the routing's choice for one token.
#pragma once
#include "common.cuh"

namespace hmoe {

// Order-preserving map of fp32 to uint32 (a > b exactly when key(a) >
// key(b)), with -0 mapped like +0 so that the two compare equal, as they do
// as floats. NaN logits are not supported.
__device__ __forceinline__ uint32_t route_key(float v) {
  uint32_t u = __float_as_uint(v);
  if ((u << 1) == 0u) u = 0u;
  return (u & 0x80000000u) ? ~u : (u | 0x80000000u);
}
__device__ __forceinline__ float route_key_value(uint32_t key) {
  return __uint_as_float((key & 0x80000000u) ? (key & 0x7FFFFFFFu) : ~key);
}

// One warp routes one token. Lane l holds logits of experts l, l+32, ...
// (E <= 512, so at most 16 per lane), as order-preserving keys. Each of the
// k rounds takes the lane's best remaining candidate (the lowest expert id
// among equal keys), then the warp's largest key and, among the lanes that
// hold it, the lowest expert id (two warp reductions), so the winners come
// in descending order with ties to the lower id. Lane r (r < k) returns the
// r-th winner's id and gate.
__device__ __forceinline__ void warp_route_token(const float* __restrict__ row, int E, int k, int lane,
                                                 int* my_id, float* my_gate) {
  uint32_t key[MAX_E / 32];
#pragma unroll
  for (int j = 0; j < MAX_E / 32; ++j) {
    const int e = lane + 32 * j;
    key[j] = (e < E) ? route_key(row[e]) : 0u;  // 0: below every real key
  }
  uint32_t taken = 0;
  int rid = 0;
  uint32_t rkey = 0;
  for (int r = 0; r < k; ++r) {
    uint32_t bk = 0;
    uint32_t be = 0xFFFFFFFFu;
#pragma unroll
    for (int j = 0; j < MAX_E / 32; ++j) {
      if (!((taken >> j) & 1u) && key[j] > bk) {  // j ascending: the first of equal keys has the lowest id
        bk = key[j];
        be = (uint32_t)(lane + 32 * j);
      }
    }
    const uint32_t m = __reduce_max_sync(0xffffffffu, bk);
    const uint32_t w = __reduce_min_sync(0xffffffffu, bk == m ? be : 0xFFFFFFFFu);
    if ((int)(w & 31u) == lane) taken |= 1u << (w >> 5);
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

}  // namespace hmoe
