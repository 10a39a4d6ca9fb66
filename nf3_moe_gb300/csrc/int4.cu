// int4.cu -- y = W x (+ bias) for few rows x and W of 4-bit integers with a scale (and a zero point) per group along K.
//
//   W[n][k] = (q[n][k] - z[n][k / G]) * s[n][k / G],  q, z in 0..15, G = 32, 64 or 128
//
// What bounds it is the bytes of W (0.516 a weight at G = 128), then, below some
// megabytes, the chain launch, loads, sums. The work is a list of units, 16 rows
// over the whole K; each CTA takes an even run of them, and its warps even
// parts of the run's k-blocks (128 of K), whole units or not. Where shared memory
// does not hold x's rows over all of K, K is taken in parts and the units' sums
// wait in shared memory (16 rows of K = 6144 in two parts: 25 us for 12288 x 6144,
// against 30 with two passes of 8 rows over the weights). A warp streams its
// blocks with cp.async into a ring of its own, decodes in registers and issues
// m16n8k16 MMAs with x's rows as the N side; the sums of a unit that several
// warps share are joined through shared memory in the order of K.
//
// Decoding. A nibble OR-ed into the low mantissa bits of 128 (bf16) or 1024 (fp16)
// is 128 + q or 1024 + q, exactly (the magic-number conversion of Kim et al., Who
// Says Elephants Can't Run: Bringing Large Scale MoE Models into Cloud Scale
// Production, 2022); 128 + z or 1024 + z is subtracted, exactly, before the
// product, 11 operations for 8 weights. The products are of (q - z) x alone, so
// that a large x on a weight of zero adds nothing. (bf16 products of 128 + q with
// the group's sum of x times 128 + z taken off afterwards are 7 operations, 25.2
// against 27.4 us for 8 rows of 32768 x 6144, 105 MB, but leave 2^-17 of the
// sum of |x s|: one x 10^6 times the others cost 13% of a result it has no part in.)
// What bounds it after the bytes is the issue of instructions and the ALU. A mask and
// an OR apart in the decoder cost 29.6 against 25.1, when that was all of it. More
// warps (20, 24) were slower, as were 8.
#include "act.cuh"
#include "common.cuh"
#include "internal.h"

namespace hmoe {

// Warps of a CTA: 16, or 8 where a CTA has few blocks, whose time is the start, the joining and the fetch of the code, and,
// with more than two rows, filling x. us with 16 warps and with 8, by the blocks of a CTA:
//   1 row:   16: 3.9, 3.2   32: 4.5, 4.2   48: 5.5, 5.3   64: 6.3, 6.1   96: 6.9, 7.1   144: 8.6, 9.0   288: 13.1, 14.9
//   2 rows:  16: 4.0, 3.3   32: 4.7, 4.6   48: 5.8, 5.6   64: 5.8, 5.9   96: 7.0, 7.5
//   3 rows:  16: 4.0, 3.7   25: 4.6, 4.8   32: 4.7, 5.0   48: 6.1, 6.3
//   8 rows:   8: 3.7, 3.3   16: 4.4, 4.4   25: 5.4, 6.1   48: 7.5, 8.5   96: 8.8, 10.4
// The rings of 8 warps also leave room for twice the x. Where those of 16 do not leave it all of K:
//   12 rows: 48: 13.8, 10.8   96: 14.3, 12.9   128: 20.0, 18.7
//   16 rows: 32: 11.5, 9.4   48: 16.9, 14.9   64: 11.3, 10.8   96: 16.6, 16.8   128: 21.5, 21.3   144: 17.9, 19.6
constexpr int I4_WARPS = 16, I4_FEW_WARPS = 8;
constexpr int I4_FEW_BLOCKS = 16, I4_FEW_BLOCKS_2ROWS = 48, I4_FEW_BLOCKS_PARTS = 128;  // at most
constexpr int I4_RING = 6;  // blocks of a warp's ring, in pairs
constexpr int I4_ROWS = 16; // rows of x of a pass
constexpr int I4_UNITS = 16;  // units worked on at once where K is taken in parts

// ------------------------------------------------------------ packing
// A block is 16 rows x 128 K. Codes: two halves of 64 K, each [32 lanes][4 words]: lane (g, q) holds rows g and g + 8
// (words 0, 1 and 2, 3); word h covers the k16 steps 2h and 2h + 1 of the half, in which a lane's values are
// k = 16 step + 4 q + 0..3: nibbles 0, 4 and 1, 5 are the first step's, 2, 6 and 3, 7 the second's. Then the scales,
// [group of the block][g][row g, row g + 8], and in the same order the zero points, a byte each.
__global__ void int4_pack_kernel(const uint8_t* __restrict__ codes, const uint16_t* __restrict__ scales,
                                 const uint8_t* __restrict__ zeros, int N, int K, int group, uint8_t* __restrict__ dst) {
  const int NB = (K + 127) / 128, ng = 128 / group, groups = K / group;
  const int unit = blockIdx.x, b = blockIdx.y, tid = threadIdx.x;
  uint8_t* blk = dst + ((size_t)unit * NB + b) * i4_block_bytes(ng, zeros != nullptr);
  {
    const int half = tid >> 7, lane = (tid >> 2) & 31, word = tid & 3;
    const int n = unit * 16 + (lane >> 2) + (word >> 1) * 8;
    uint32_t v = 0;
    if (n < N)
      for (int i = 0; i < 8; ++i) {
        const int step = 2 * (word & 1) + ((i >> 1) & 1), e = 2 * (i & 1) + (i >> 2);
        const int k = b * 128 + half * 64 + step * 16 + (lane & 3) * 4 + e;
        // nibble position of element e of the step: pairs (0, 4), (1, 5) for even steps, (2, 6), (3, 7) for odd ones
        const int at = 2 * (step & 1) + (e >> 1) + 4 * (e & 1);
        if (k < K) v |= (uint32_t)((codes[(size_t)n * (K / 2) + k / 2] >> (4 * (k & 1))) & 15u) << (4 * at);
      }
    reinterpret_cast<uint32_t*>(blk)[half * 128 + lane * 4 + word] = v;
  }
  if (tid < ng * 16) {
    const int gr = tid >> 4, g = (tid >> 1) & 7, n = unit * 16 + g + (tid & 1) * 8, at = b * ng + gr;
    const bool there = n < N && at < groups;
    reinterpret_cast<uint16_t*>(blk + 1024)[tid] = there ? scales[(size_t)n * groups + at] : 0;
    if (zeros) blk[1024 + ng * 32 + tid] = there ? (zeros[(size_t)n * groups + at] & 15) : 0;
  }
}

cudaError_t launch_int4_pack(const Int4Geom& g, const uint8_t* codes, const uint16_t* scales, const uint8_t* zeros,
                             uint8_t* dst, cudaStream_t st) {
  int4_pack_kernel<<<dim3(g.units, g.NB), 256, 0, st>>>(codes, scales, zeros, g.N, g.K, g.group, dst);
  count_launches(1);
  return cudaGetLastError();
}

// ------------------------------------------------------------ product
template <int ACT>
__device__ __forceinline__ uint32_t sub_x2(uint32_t a, uint32_t b) {
  uint32_t d;
  if constexpr (ACT == ACT_F16) asm("sub.rn.f16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
  else asm("sub.rn.bf16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
  return d;
}
// (v & mask) | bits in one operation: both as registers, since as constants the compiler takes an operation for each.
__device__ __forceinline__ uint32_t and_or(uint32_t v, uint32_t mask, uint32_t bits) {
  uint32_t d;
  asm("lop3.b32 %0, %1, %2, %3, 0xEA;" : "=r"(d) : "r"(v), "r"(mask), "r"(bits));
  return d;
}
template <int ACT>
__device__ __forceinline__ float act_lo(uint32_t v) { return act_x2_to_f32<ACT>(v).x; }

template <int ACT, int NT, int NG, int WARPS>
__global__ void __launch_bounds__(WARPS * 32, 1) int4_kernel(const __grid_constant__ Int4Params p) {
  extern __shared__ __align__(128) uint8_t smem[];
  constexpr uint32_t MAGIC = ACT == ACT_F16 ? 0x64006400u : 0x43004300u;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, g = lane >> 2, q = lane & 3;
  const int BB = i4_block_bytes(NG, p.zeros != 0), NB = p.NB;
  // not constants to the compiler
  const uint32_t mask = p.mask, magic = p.magic;
  uint8_t* const ring = smem + warp * I4_RING * BB;
  float* const part = reinterpret_cast<float*>(smem + WARPS * I4_RING * BB);  // [warps][4 NT][32]
  float* const kept = part + WARPS * 4 * NT * 32;  // K in parts: [I4_UNITS][4 NT][32]
  uint8_t* const xs = reinterpret_cast<uint8_t*>(kept + (p.parts > 1 ? I4_UNITS * 4 * NT * 32 : 0));
  const int t0 = blockIdx.y * p.pass, nt = min(p.pass, p.T - t0);
  const int u0 = div_by(p.units * (int)blockIdx.x, p.by_grid), u1 = div_by(p.units * ((int)blockIdx.x + 1), p.by_grid);
  const int pieces = BB / 16 - 64;  // of a block's scales and zero points
  const uint32_t dst0 = smem_u32(ring) + lane * 16;
  const int half = nt * 64;
  const uint8_t* const x0 = xs + g * 64 + q * 16;
  const bool on0 = g < nt, on1 = 8 + g < nt;

  // Now: units [ub, ub + nu), part c of K, nb blocks from block c * kc on; this warp's steps (blocks) of them.
  int ub = u0, c = 0, nu = p.parts > 1 ? min(I4_UNITS, u1 - u0) : u1 - u0, nb = p.parts > 1 ? p.kc : NB;
  auto by_nb = [&](int n) { return c == p.parts - 1 ? div_by(n, p.by_last) : div_by(n, p.by_kc); };
  auto border = [&](int w) { return (int)((long long)(nu * nb) * w / WARPS); };
  int from = 0, to = 0, unit = 0, st = 0, slot = 0, ahead = 0, left = 0;
  const uint8_t* at = p.packed;  // this lane's 16 bytes of the next block to copy: a unit's blocks, and units, lie one after another
  bool whole = true;
  auto copy = [&](int s) {
    const uint32_t dst = dst0 + s * BB;
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(at) : "memory");
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst + 512), "l"(at + 512) : "memory");
    if (lane < pieces) asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst + 1024), "l"(at + 1024) : "memory");
    at += BB;
    if (--left == 0) {  // the unit's blocks of this part of K
      left = nb;
      at += (size_t)(NB - nb) * BB;
    }
  };
  auto copy2 = [&](int s) {
    if (ahead < to) copy(s);
    if (ahead + 1 < to) copy(s + 1);
    ahead += 2;
    asm volatile("cp.async.commit_group;" ::: "memory");
  };
  auto place = [&]() {
    from = border(warp);
    to = border(warp + 1);
    unit = by_nb(from);
    st = from - unit * nb;
    slot = 0;
    ahead = from;
    left = nb - st;
    whole = st == 0;
    at = p.packed + ((size_t)(ub + unit) * NB + (size_t)c * p.kc + st) * BB + lane * 16;
  };
  place();
  // The first weights to L2 while the kernel before still runs; nothing is read before the wait.
  for (int i = lane; i < min(I4_RING - 2, min(to - from, left)) * (BB / 128); i += 32)
    asm volatile("prefetch.global.L2 [%0];" ::"l"(at - lane * 16 + i * 128));
  pdl_wait();
  pdl_trigger();

  float acc[NT][4] = {};
  auto clear = [&]() {
#pragma unroll
    for (int i = 0; i < 4 * NT; ++i) acc[i >> 2][i & 3] = 0.0f;
  };
  // The sums of unit ub + u over this part of K: kept for the next part, or the result.
  auto finish = [&](int u) {
    if (p.parts > 1) {
      float* k = kept + (u * 4 * NT) * 32 + lane;
#pragma unroll
      for (int i = 0; i < 4 * NT; ++i) {
        if (c > 0) acc[i >> 2][i & 3] += k[i * 32];
        if (c < p.parts - 1) k[i * 32] = acc[i >> 2][i & 3];
      }
      if (c < p.parts - 1) return;
    }
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int col = 8 * n + 2 * q + (i & 1), r = (ub + u) * 16 + g + (i >> 1) * 8;
        if (col < nt && r < p.N) {
          const float b = p.bias ? act_lo<ACT>((uint32_t)p.bias[r]) : 0.0f;
          p.out[(size_t)(t0 + col) * p.ldout + r] = f32_to_act<ACT>(acc[n][i] + b);
        }
      }
  };
  const uint8_t *x = x0, *w = ring;
  auto block = [&]() {
    float d[NT][4];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const uint4 c4 = reinterpret_cast<const uint4*>(w)[h * 32 + lane];
      const uint32_t cw[4] = {c4.x, c4.y, c4.z, c4.w};
      uint4 xv[NT][2];
#pragma unroll
      for (int n = 0; n < NT; ++n)
        if (n ? on1 : on0) {
          xv[n][0] = *reinterpret_cast<const uint4*>(x + n * 512);
          xv[n][1] = *reinterpret_cast<const uint4*>(x + n * 512 + half);
        }
      x += 2 * half;
#pragma unroll
      for (int k = 0; k < 2; ++k) {  // two k16 steps
        const int gr = NG == 4 ? 2 * h + k : (NG == 2 ? h : 0);
        const bool begin = NG == 4 || (k == 0 && (NG == 2 || h == 0)), end = NG == 4 || (k == 1 && (NG == 2 || h == 1));
        uint32_t z = 0x0808u;  // of row g, and of row g + 8
        if (p.zeros) z = *reinterpret_cast<const uint16_t*>(w + 1024 + NG * 32 + gr * 16 + g * 2);
        uint32_t a[2][4];  // pairs of row g and of row g + 8
#pragma unroll
        for (int r = 0; r < 2; ++r)
#pragma unroll
          for (int i = 0; i < 4; ++i)
            a[r][i] = sub_x2<ACT>(and_or(cw[2 * r + k] >> (4 * i), mask, magic), (r ? z >> 8 : z & 0xFFu) * 0x00010001u + MAGIC);
#pragma unroll
        for (int n = 0; n < NT; ++n) {
          const uint4& xk = xv[n][k];
          if (begin) mma_16816_zc<ACT>(d[n], a[0][0], a[1][0], a[0][1], a[1][1], xk.x, xk.y);
          else mma_16816<ACT>(d[n], a[0][0], a[1][0], a[0][1], a[1][1], xk.x, xk.y);
          mma_16816<ACT>(d[n], a[0][2], a[1][2], a[0][3], a[1][3], xk.z, xk.w);
        }
        if (end) {
          const float2 sc = act_x2_to_f32<ACT>(*reinterpret_cast<const uint32_t*>(w + 1024 + gr * 32 + g * 4));
#pragma unroll
          for (int n = 0; n < NT; ++n) {
            acc[n][0] = fmaf(sc.x, d[n][0], acc[n][0]);
            acc[n][1] = fmaf(sc.x, d[n][1], acc[n][1]);
            acc[n][2] = fmaf(sc.y, d[n][2], acc[n][2]);
            acc[n][3] = fmaf(sc.y, d[n][3], acc[n][3]);
          }
        }
      }
    }
    w += BB;
    if (++st == nb) {
      if (whole) {
        finish(unit);
      } else {
#pragma unroll
        for (int i = 0; i < 4 * NT; ++i) part[(warp * 4 * NT + i) * 32 + lane] = acc[i >> 2][i & 3];
      }
      clear();
      whole = true;
      st = 0;
      x = x0;
      ++unit;
    }
  };
  for (;;) {
#pragma unroll 1
    for (int i = 0; i < I4_RING - 2; i += 2) copy2(i);
    // x as fragments: [64 of K][half][row][q], 16 bytes: the q-th four values of the half's two k16 steps. A thread
    // has 8 values. The loads are coherent ones, since the kernel before may write x while this one starts. Few blocks: less code to fetch (one row of 2048 x 2048:
    // 3.2 us with two loads in flight, 3.4 with four; 8 rows of 32768 x 6144: 26.4 and 25.0).
    {
      constexpr int LOADS = WARPS == I4_FEW_WARPS ? 2 : 4;
      const int chunks = nb * 16, all = chunks * nt, k0 = c * p.kc * 16;
      for (int i0 = tid; i0 < all; i0 += LOADS * (WARPS * 32)) {
        uint4 v[LOADS];
#pragma unroll
        for (int j = 0; j < LOADS; ++j) {
          const int i = i0 + j * (WARPS * 32), r = by_nb(min(i, all - 1)) >> 4, k = k0 + i - r * chunks;
          v[j] = i < all && k * 8 < p.K ? __ldca(reinterpret_cast<const uint4*>(p.x + (size_t)(t0 + r) * p.ldx) + k) : make_uint4(0, 0, 0, 0);
        }
#pragma unroll
        for (int j = 0; j < LOADS; ++j) {
          const int i = i0 + j * (WARPS * 32), r = by_nb(min(i, all - 1)) >> 4, k = i - r * chunks;
          if (i < all) {
            const int step = (k >> 1) & 3;
            uint8_t* d = xs + (((k >> 3) * 2 + (step >> 1)) * nt + r) * 64 + (k & 1) * 32 + (step & 1) * 8;
            *reinterpret_cast<uint2*>(d) = make_uint2(v[j].x, v[j].y);
            *reinterpret_cast<uint2*>(d + 16) = make_uint2(v[j].z, v[j].w);
          }
        }
      }
    }
    __syncthreads();
    x = x0 + st * 4 * half;
    w = ring;
    for (int s = from; s < to; s += 2) {
      asm volatile("cp.async.wait_group %0;" ::"n"(I4_RING / 2 - 2) : "memory");
      __syncwarp();
      copy2(slot == 0 ? I4_RING - 2 : slot - 2);  // into the pair before, which all lanes have read
      block();
      if (s + 1 < to) block();
      slot += 2;
      if (slot == I4_RING) {
        slot = 0;
        w = ring;
      }
    }
    __syncwarp();
    float* const rest = reinterpret_cast<float*>(ring);  // the sums of a unit that another warp ends
    if (st != 0 && from < to)
#pragma unroll
      for (int i = 0; i < 4 * NT; ++i) rest[i * 32 + lane] = acc[i >> 2][i & 3];
    __syncthreads();
    // The unit that this warp ended and others began, in the order of K.
    const int mine = by_nb(from), begin = mine * nb;
    if (from != begin && to >= begin + nb) {
      int v = warp - 1;
      while (border(v) > begin) --v;
      clear();
      for (; v < warp; ++v) {
        if (border(v) == border(v + 1)) continue;  // a warp without work
        const float* theirs = reinterpret_cast<const float*>(smem + v * I4_RING * BB);
#pragma unroll
        for (int i = 0; i < 4 * NT; ++i) acc[i >> 2][i & 3] += theirs[i * 32 + lane];
      }
#pragma unroll
      for (int i = 0; i < 4 * NT; ++i) acc[i >> 2][i & 3] += part[(warp * 4 * NT + i) * 32 + lane];
      finish(mine);
    }
    if (p.parts == 1) return;
    if (++c == p.parts) {
      c = 0;
      ub += nu;
      if (ub >= u1) return;
      nu = min(I4_UNITS, u1 - ub);
    }
    nb = c == p.parts - 1 ? NB - c * p.kc : p.kc;
    clear();
    place();
    __syncthreads();  // the rings, the sums and x are free
  }
}

// ------------------------------------------------------------ launch
// Bytes of shared memory beside x for passes of `pass` rows.
static int i4_fixed(int ng, int pass, bool parts, int warps) {
  const int nt = pass > 8 ? 2 : 1;
  return warps * (I4_RING * i4_block_bytes(ng, true) + nt * 512) + (parts ? I4_UNITS * nt * 512 : 0);
}

template <int ACT, int NT, int NG, int WARPS>
static cudaError_t launch_as(const Int4Params& p, dim3 grid, int smem, cudaStream_t st) {
  static std::atomic<unsigned long long> attr{0};
  const cudaError_t e = ensure_smem_attr(int4_kernel<ACT, NT, NG, WARPS>, DK_SMEM_LIMIT, attr);
  return e != cudaSuccess ? e : launch_pdl(int4_kernel<ACT, NT, NG, WARPS>, grid, dim3(WARPS * 32), (size_t)smem, st, p);
}
template <int ACT, int NT, int WARPS>
static cudaError_t launch_by_group(const Int4Params& p, int ng, dim3 grid, int smem, cudaStream_t st) {
  return ng == 1 ? launch_as<ACT, NT, 1, WARPS>(p, grid, smem, st)
                 : (ng == 2 ? launch_as<ACT, NT, 2, WARPS>(p, grid, smem, st) : launch_as<ACT, NT, 4, WARPS>(p, grid, smem, st));
}
template <int ACT>
static cudaError_t launch_by_size(const Int4Params& p, int nt, bool few, int ng, dim3 grid, int smem, cudaStream_t st) {
  if (few) return nt == 2 ? launch_by_group<ACT, 2, I4_FEW_WARPS>(p, ng, grid, smem, st) : launch_by_group<ACT, 1, I4_FEW_WARPS>(p, ng, grid, smem, st);
  return nt == 2 ? launch_by_group<ACT, 2, I4_WARPS>(p, ng, grid, smem, st) : launch_by_group<ACT, 1, I4_WARPS>(p, ng, grid, smem, st);
}

cudaError_t launch_int4(Int4Params p, int ng, int num_sms, cudaStream_t st) {
  const int passes = (p.T + I4_ROWS - 1) / I4_ROWS;
  p.pass = (p.T + passes - 1) / passes;  // the passes evened out
  const int nt = p.pass > 8 ? 2 : 1, per = p.pass * 256;  // bytes of x for each block of K
  const unsigned ctas = (unsigned)(p.units < num_sms ? p.units : num_sms);
  const auto in_parts = [&](int w) { return p.NB * per > DK_SMEM_LIMIT - i4_fixed(ng, p.pass, false, w); };
  const int most_few = in_parts(I4_WARPS) ? I4_FEW_BLOCKS_PARTS : (p.pass <= 2 ? I4_FEW_BLOCKS_2ROWS : I4_FEW_BLOCKS);
  const bool few = (long long)((p.units + (int)ctas - 1) / (int)ctas) * p.NB <= most_few;
  const int warps = few ? I4_FEW_WARPS : I4_WARPS;
  p.parts = 1;
  if (in_parts(warps)) {
    const int most = (DK_SMEM_LIMIT - i4_fixed(ng, p.pass, true, warps)) / per;
    p.parts = (p.NB + most - 1) / most;
  }
  p.kc = (p.NB + p.parts - 1) / p.parts;
  p.parts = (p.NB + p.kc - 1) / p.kc;  // none empty
  p.by_kc = div_by_const((uint32_t)p.kc);
  p.by_last = div_by_const((uint32_t)(p.NB - (p.parts - 1) * p.kc));
  const int smem = i4_fixed(ng, p.pass, p.parts > 1, warps) + p.kc * per;
  const dim3 grid(ctas, (unsigned)passes);
  p.by_grid = div_by_const(grid.x);
  p.mask = 0x000F000Fu;
  p.magic = p.act_type == ACT_F16 ? 0x64006400u : 0x43004300u;
  const cudaError_t e = p.act_type == ACT_F16 ? launch_by_size<ACT_F16>(p, nt, few, ng, grid, smem, st)
                                              : launch_by_size<ACT_BF16>(p, nt, few, ng, grid, smem, st);
  count_launches(1);
  return e;
}

}  // namespace hmoe
