// dispatch.cu -- token rows sorted by expert and back, with the gates applied, and their gradients.
//
// With s = t * topk + j a slot, slot_row[s] its row in the sorted buffer (or
// none) and row_slot the inverse map:
//   dispatch   rows[r] = (g[s]) x[s / topk], s = row_slot[r]; pad rows are zero
//   combine    out[t] = sum_j (g[t,j]) rows[slot_row[t,j]]
// The gradient of each is the other, plus the gates' part:
//   combine:   drows[r] = (g[s]) dout[s / topk],     dg[s] = <rows[slot_row[s]], dout[t]>
//   dispatch:  dx[t] = sum_j (g[t,j]) drows[slot_row[t,j]], dg[s] = <drows[slot_row[s]], x[t]>
// and through the softmax over the chosen experts
//   dlogits[t, ids[t,j]] = g_j (dg_j - sum_i g_i dg_i), zero elsewhere.
// So two kernels do the data movement: spread (tokens to rows) and collect
// (rows to tokens), each with the dot products of the gates' gradient as an
// option. Every sum is fp32 in a fixed order; a slot without a row takes no
// part (it is skipped, not multiplied by zero, so what pad rows hold never
// reaches a result).
//
// HBM bounds them all from some hundred rows on. At 4096 tokens of 6144 16-bit
// columns, 256 experts, top-8 (of the copy bandwidth 6.70 TB/s):
//   dispatch, with its plan      453 MB   73.4 us   92%
//   combine                      453 MB   67.3 us   100%
//   combine's gradient, with the gates' and logits', 860 MB, 131 us, 98%
// Small batches are a launch or two: 8 tokens dispatched in 3.3 us, one token
// combined in 2.3 us.
#include "act.cuh"
#include "common.cuh"
#include "internal.h"

namespace hmoe {

// ------------------------------------------------------------ element types
constexpr int ROW_BF16 = 0, ROW_F16 = 1, ROW_F32 = 2;

template <int DT>
struct Elem;
template <>
struct Elem<ROW_BF16> {
  using type = uint16_t;
};
template <>
struct Elem<ROW_F16> {
  using type = uint16_t;
};
template <>
struct Elem<ROW_F32> {
  using type = float;
};
template <int DT>
__device__ __forceinline__ float to_f32(typename Elem<DT>::type v) {
  if constexpr (DT == ROW_F32) return v;
  else if constexpr (DT == ROW_F16) return __half2float(__ushort_as_half(v));
  else return bf16_bits_to_float(v);
}
template <int DT>
__device__ __forceinline__ typename Elem<DT>::type from_f32(float f) {
  if constexpr (DT == ROW_F32) return f;
  else if constexpr (DT == ROW_F16) return f32_to_act<ACT_F16>(f);
  else return f32_to_act<ACT_BF16>(f);
}

// A piece of a row: 16 bytes where the width and the addresses allow it (VEC),
// else 4 elements, as far apart as the row has threads, so that a warp's accesses
// stay side by side and each thread has 4 on their way (3000 tokens of 999 16-bit
// columns, top-2, and one element at a time: dispatch 7.5 and 15.7 us, combine
// 8.8 and 10.3, their gradients 12.6 and 18.4, 14.6 and 21.6).
template <int DT, bool VEC>
struct Piece {
  using E = typename Elem<DT>::type;
  static constexpr int N = VEC ? 16 / (int)sizeof(E) : 4;
  // Where a thread's piece begins among `threads` that share a row, and how far
  // they get together.
  static __device__ __forceinline__ int first(int part, int threads, int tid) {
    return VEC ? (part * threads + tid) * N : part * threads * N + tid;
  }
  E v[N];
  // p: the first element; threads: of the row; left: elements from the first to
  // the row's end. Elements past it read as zero.
  __device__ __forceinline__ void load(const E* p, int threads, int left) {
    if constexpr (VEC) *reinterpret_cast<uint4*>(v) = *reinterpret_cast<const uint4*>(p);
    else
#pragma unroll
      for (int i = 0; i < N; ++i) v[i] = i * threads < left ? p[i * threads] : E(0);
  }
  __device__ __forceinline__ void store(E* p, int threads, int left) const {
    if constexpr (VEC) *reinterpret_cast<uint4*>(p) = *reinterpret_cast<const uint4*>(v);
    else
#pragma unroll
      for (int i = 0; i < N; ++i)
        if (i * threads < left) p[i * threads] = v[i];
  }
  // For rows that pass through once: they leave L2 before what is kept.
  __device__ __forceinline__ void load_once(const E* p, int threads, int left) {
    if constexpr (VEC) *reinterpret_cast<uint4*>(v) = __ldcs(reinterpret_cast<const uint4*>(p));
    else
#pragma unroll
      for (int i = 0; i < N; ++i) v[i] = i * threads < left ? __ldcs(p + i * threads) : E(0);
  }
  __device__ __forceinline__ void store_once(E* p, int threads, int left) const {
    if constexpr (VEC) __stcs(reinterpret_cast<uint4*>(p), *reinterpret_cast<const uint4*>(v));
    else
#pragma unroll
      for (int i = 0; i < N; ++i)
        if (i * threads < left) __stcs(p + i * threads, v[i]);
  }
  __device__ __forceinline__ float f(int i) const { return to_f32<DT>(v[i]); }
  __device__ __forceinline__ void set(int i, float x) { v[i] = from_f32<DT>(x); }
};

// ------------------------------------------------------------ the row maps
// Expert e keeps its first min(n_e, capacity) slots (capacity 0: all) in
// ascending slot order; its rows start at row_offsets[e], a multiple of
// align. Every CTA scans the E counts itself (E <= 512: one value a thread),
// then takes its share of the rows and, with a capacity, of the slots.
struct DispatchPlan {
  const int* perm;
  const int* offsets;
  int S, E, align, capacity, R;
  int* row_slot;
  int* slot_row;
  int* row_offsets;
  int* status;
};
struct PlanScan {
  int off[MAX_E], n[MAX_E], row[MAX_E + 1], warp[MAX_E / 32];
};
// All MAX_E threads; ends with a barrier. The first CTA writes row_offsets.
__device__ __forceinline__ void plan_scan(const DispatchPlan& p, PlanScan& s) {
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  int n = 0, o = 0;
  bool bad = false;
  if (tid < p.E) {
    // perm is indexed with these, so they are clamped to it.
    const int a = p.offsets[tid], b = p.offsets[tid + 1];
    bad = a < 0 || b < a || b > p.S || (tid == 0 && a != 0) || (tid == p.E - 1 && b != p.S);
    o = min(max(a, 0), p.S);
    n = max(min(b, p.S) - o, 0);
    if (p.capacity > 0) n = min(n, p.capacity);
  }
  if (bad) set_status(p.status, DEV_BAD_ROUTE);
  const int padded = (int)(((long long)n + p.align - 1) / p.align) * p.align;
  int incl = padded;
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const int v = __shfl_up_sync(0xffffffffu, incl, d);
    if (lane >= d) incl += v;
  }
  if (lane == 31) s.warp[warp] = incl;
  __syncthreads();
  int before = 0;
  for (int w = 0; w < warp; ++w) before += s.warp[w];
  const int start = before + incl - padded;
  if (tid < p.E) {
    s.off[tid] = o;
    s.n[tid] = n;
    s.row[tid] = start;
    if (tid == p.E - 1) s.row[p.E] = start + padded;
    if (blockIdx.x == 0) {
      p.row_offsets[tid] = min(start, p.R);
      if (tid == p.E - 1) p.row_offsets[p.E] = min(start + padded, p.R);
    }
  }
  __syncthreads();
}
// The slot of row r, or -1.
__device__ __forceinline__ int plan_row(const DispatchPlan& p, const PlanScan& s, int r) {
  if (r >= s.row[p.E]) return -1;
  int lo = 0, hi = p.E - 1;  // the last expert that starts at or before r
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (s.row[mid] <= r) lo = mid;
    else hi = mid - 1;
  }
  const int rank = r - s.row[lo];
  if (rank < 0 || rank >= s.n[lo]) return -1;
  const int slot = p.perm[s.off[lo] + rank];
  if (slot < 0 || slot >= p.S) {
    set_status(p.status, DEV_BAD_ROUTE);
    return -1;
  }
  return slot;
}
// With a capacity: -1 for the slots that it drops. All threads of the grid.
// Rows and slots go up to INT_MAX, so the counters that step by a grid past
// them are unsigned.
__device__ __forceinline__ void plan_dropped(const DispatchPlan& p, const PlanScan& s) {
  if (p.capacity <= 0) return;
  for (unsigned at = blockIdx.x * blockDim.x + threadIdx.x; at < (unsigned)p.S; at += gridDim.x * blockDim.x) {
    const int i = (int)at;
    int lo = 0, hi = p.E - 1;
    while (lo < hi) {
      const int mid = (lo + hi + 1) >> 1;
      if (s.off[mid] <= i) lo = mid;
      else hi = mid - 1;
    }
    const int slot = p.perm[i];
    if (i - s.off[lo] >= s.n[lo] && slot >= 0 && slot < p.S) p.slot_row[slot] = -1;
  }
}

__global__ void __launch_bounds__(MAX_E) dispatch_plan_kernel(DispatchPlan p) {
  __shared__ PlanScan s;
  pdl_wait();
  pdl_trigger();
  plan_scan(p, s);
  for (unsigned r = blockIdx.x * blockDim.x + threadIdx.x; r < (unsigned)p.R; r += gridDim.x * blockDim.x) {
    const int slot = plan_row(p, s, (int)r);
    p.row_slot[r] = slot;
    if (slot >= 0) p.slot_row[slot] = (int)r;
  }
  plan_dropped(p, s);
}

// Small batches: the plan and the rows in one launch, a CTA a row. A row of x
// is read once for each of its slots, which L2 serves.
template <int DT, bool VEC>
__global__ void __launch_bounds__(MAX_E) dispatch_small_kernel(DispatchPlan p, RowsParams q) {
  using P = Piece<DT, VEC>;
  using E = typename P::E;
  __shared__ PlanScan s;
  __shared__ int s_slot;
  pdl_wait();
  pdl_trigger();
  plan_scan(p, s);
  const int tid = threadIdx.x;
  for (int r = blockIdx.x; r < p.R; r += gridDim.x) {
    if (tid == 0) {
      const int slot = plan_row(p, s, r);
      p.row_slot[r] = slot;
      if (slot >= 0) p.slot_row[slot] = r;
      s_slot = slot;
    }
    __syncthreads();
    const int slot = s_slot;
    const E* v = static_cast<const E*>(q.v) + (size_t)(max(slot, 0) / q.topk) * q.H;
    E* dst = static_cast<E*>(q.rows_out) + (size_t)r * q.H;
    const float g = q.gates && slot >= 0 ? q.gates[slot] : 1.0f;
    for (int c = P::first(0, MAX_E, tid); c < q.H; c += MAX_E * P::N) {
      P a;
      if (slot >= 0) {
        a.load(v + c, MAX_E, q.H - c);
        if (q.gates) {
#pragma unroll
          for (int i = 0; i < P::N; ++i) a.set(i, g * a.f(i));
        }
      } else {
#pragma unroll
        for (int i = 0; i < P::N; ++i) a.set(i, 0.0f);
      }
      a.store(dst + c, MAX_E, q.H - c);
    }
    __syncthreads();
  }
  plan_dropped(p, s);
}

// ------------------------------------------------------------ the gates' gradient of one token
// dg, g, ids: the token's topk dot products, gates and experts, in shared
// memory. Called by nthreads threads; no barrier inside.
__device__ __forceinline__ void write_gate_grads(const float* dg, const float* g, const int* ids, int t, int k, int E,
                                                 float* dgates, float* dlogits, int tid, int nthreads, int* status) {
  if (dgates && tid < k) dgates[(size_t)t * k + tid] = dg[tid];
  if (!dlogits) return;
  float mean = 0.0f;  // sum_i g_i dg_i, ascending i
  for (int j = 0; j < k; ++j) mean = fmaf(g[j], dg[j], mean);
  for (int e = tid; e < E; e += nthreads) {
    float v = 0.0f;
    for (int j = 0; j < k; ++j)
      if (ids[j] == e) v = g[j] * (dg[j] - mean);
    dlogits[(size_t)t * E + e] = v;
  }
  if (tid < k && (ids[tid] < 0 || ids[tid] >= E)) set_status(status, DEV_BAD_ROUTE);
}

// ------------------------------------------------------------ one token a CTA
// The columns of a token are dealt to the threads (and to the grid's y where no
// dot products need them together), 16 bytes each. A thread meets the token's
// topk rows at its columns, so each value of the token is read or written once
// and the rows' accesses are in flight together.
// Narrow rows share a CTA, each with 32, 64 or 128 of its threads.
constexpr int ROWS_THREADS = 256;
constexpr int ROWS_TOKENS = 8;  // of a CTA, at most
template <bool MANY>
struct TokenCta {
  static constexpr int TOKENS = MANY ? ROWS_TOKENS : 1;
  static __device__ __forceinline__ int threads() { return MANY ? blockDim.x : ROWS_THREADS; }  // of a token
  static __device__ __forceinline__ int tokens() { return MANY ? blockDim.y : 1; }
  static __device__ __forceinline__ int at() { return MANY ? threadIdx.y : 0; }
  static __device__ __forceinline__ int token() { return blockIdx.x * tokens() + at(); }
};

// The rows and weights of token t's slots (and, for the router's gradient, their
// experts: at the end they would be waited for), in shared memory (a barrier
// follows).
struct TokenSlots {
  int row[MAX_TOPK], id[MAX_TOPK];
  float g[MAX_TOPK];
};
template <bool IDS>
__device__ __forceinline__ void token_slots(const RowsParams& p, int t, TokenSlots& s) {
  const int j = threadIdx.x;
  if (j < p.topk && t < p.T) {
    const size_t at = (size_t)t * p.topk + j;
    int r = p.slot_row[at];
    if constexpr (IDS) s.id[j] = p.dlogits ? p.ids[at] : 0;
    s.g[j] = p.gates ? p.gates[at] : 1.0f;
    if (r >= p.R) {
      set_status(p.status, DEV_BAD_ROUTE);
      r = -1;
    }
    s.row[j] = r;
  }
}

// The tokens' dot products from the threads' parts, then their gate gradients.
template <int KD, bool MANY>
struct TokenDots {
  float part[KD][ROWS_THREADS / 32], dg[TokenCta<MANY>::TOKENS][KD];
};
template <int KD, bool MANY>
__device__ __forceinline__ void token_dots(const RowsParams& p, int t, const float* dot, TokenDots<KD, MANY>& d, const TokenSlots& s) {
  using C = TokenCta<MANY>;
  const int tid = threadIdx.x, y = C::at(), lane = tid & 31, warps = C::threads() / 32, w0 = y * warps;
#pragma unroll
  for (int j = 0; j < KD; ++j) {
    float v = dot[j];
#pragma unroll
    for (int x = 16; x > 0; x >>= 1) v += __shfl_xor_sync(0xffffffffu, v, x);
    if (lane == 0) d.part[j][w0 + (tid >> 5)] = v;
  }
  __syncthreads();
  if (tid < p.topk) {
    float v = 0.0f;
#pragma unroll
    for (int w = 0; w < ROWS_THREADS / 32; ++w)
      if (w < warps) v += d.part[tid][w0 + w];
    d.dg[y][tid] = v;
  }
  __syncthreads();
  if (t < p.T) write_gate_grads(d.dg[y], s.g, s.id, t, p.topk, p.E, p.dgates, p.dlogits, tid, C::threads(), p.status);
}

// spread: rows[slot_row[t,j]] = (g[t,j]) v[t], and with KDOT > 0 (at least topk)
// dg[t,j] = <v[t], other[slot_row[t,j]]>. The CTAs past the tokens write zeros
// to the rows without a slot.
template <int DT, bool VEC, int KDOT, bool MANY>
__global__ void __launch_bounds__(ROWS_THREADS) spread_kernel(RowsParams p) {
  using P = Piece<DT, VEC>;
  using E = typename P::E;
  constexpr int KD = KDOT > 0 ? KDOT : 1;
  using C = TokenCta<MANY>;
  __shared__ TokenSlots s_slots[C::TOKENS];
  __shared__ TokenDots<KD, MANY> s_dots;
  pdl_wait();
  pdl_trigger();
  const int tid = threadIdx.x, lane = tid & 31;
  const int k = p.topk, t = C::token();
  const int H = p.H, threads = C::threads(), step = threads * gridDim.y * P::N;
  const unsigned blocks = ((unsigned)p.T + C::tokens() - 1) / C::tokens();  // with tokens
  TokenSlots& s = s_slots[C::at()];
  E* rows = static_cast<E*>(p.rows_out);
  if (blockIdx.x >= blocks) {
    P zero;
#pragma unroll
    for (int i = 0; i < P::N; ++i) zero.set(i, 0.0f);
    constexpr int warps = ROWS_THREADS / 32;
    const int warp = (C::at() * C::threads() + tid) / 32;
    const long long nw = (long long)(gridDim.x - blocks) * gridDim.y * warps;
    for (long long r = ((long long)(blockIdx.x - blocks) * gridDim.y + blockIdx.y) * warps + warp; r < p.R; r += nw) {
      const int slot = p.row_slot[r];
      if (slot >= 0 && slot < p.T * k) continue;
      for (int c = P::first(0, 32, lane); c < H; c += 32 * P::N) zero.store_once(rows + (size_t)r * H + c, 32, H - c);
    }
    return;
  }
  token_slots<(KDOT > 0)>(p, t, s);
  __syncthreads();
  const E* v = static_cast<const E*>(p.v) + (size_t)t * p.H;
  const E* other = static_cast<const E*>(p.other);
  float dot[KD];
#pragma unroll
  for (int j = 0; j < KD; ++j) dot[j] = 0.0f;
  for (int c = P::first(blockIdx.y, threads, tid); c < H && (!MANY || t < p.T); c += step) {
    P a;
    a.load(v + c, threads, H - c);
    if constexpr (KDOT > 0) {
#pragma unroll
      for (int j0 = 0; j0 < KDOT; j0 += 8) {
        if (j0 >= k) break;
        P b[8];
#pragma unroll
        for (int j = 0; j < 8; ++j)
          if (j0 + j < k && s.row[j0 + j] >= 0) b[j].load_once(other + (size_t)s.row[j0 + j] * H + c, threads, H - c);
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          if (j0 + j >= k || s.row[j0 + j] < 0) continue;
          const float g = s.g[j0 + j];
          P o;
#pragma unroll
          for (int i = 0; i < P::N; ++i) {
            dot[j0 + j] = fmaf(a.f(i), b[j].f(i), dot[j0 + j]);
            o.set(i, g * a.f(i));
          }
          o.store_once(rows + (size_t)s.row[j0 + j] * H + c, threads, H - c);
        }
      }
    } else {
#pragma unroll 8
      for (int j = 0; j < k; ++j) {
        const int r = s.row[j];
        if (r < 0) continue;
        P o = a;
        if (p.gates) {
#pragma unroll
          for (int i = 0; i < P::N; ++i) o.set(i, s.g[j] * a.f(i));
        }
        o.store_once(rows + (size_t)r * H + c, threads, H - c);
      }
    }
  }
  if constexpr (KDOT > 0) token_dots<KDOT>(p, t, dot, s_dots, s);
}

// collect: out[t] = sum_j (g[t,j]) rows[slot_row[t,j]], ascending j, and with
// KDOT > 0 (at least topk) dg[t,j] = <rows[slot_row[t,j]], v[t]>.
template <int DT, bool VEC, int KDOT, bool MANY>
__global__ void __launch_bounds__(ROWS_THREADS) collect_kernel(RowsParams p) {
  using P = Piece<DT, VEC>;
  using E = typename P::E;
  constexpr int KD = KDOT > 0 ? KDOT : 1;
  using C = TokenCta<MANY>;
  __shared__ TokenSlots s_slots[C::TOKENS];
  __shared__ TokenDots<KD, MANY> s_dots;
  pdl_wait();
  pdl_trigger();
  const int tid = threadIdx.x;
  const int k = p.topk, t = C::token();
  const int H = p.H, threads = C::threads();
  TokenSlots& s = s_slots[C::at()];
  token_slots<(KDOT > 0)>(p, t, s);
  __syncthreads();
  const E* rows = static_cast<const E*>(p.rows_in);
  E* out = static_cast<E*>(p.out) + (size_t)t * p.H;
  const E* v = KDOT ? static_cast<const E*>(p.v) + (size_t)t * p.H : nullptr;
  float dot[KD];
#pragma unroll
  for (int j = 0; j < KD; ++j) dot[j] = 0.0f;
  for (int c = P::first(blockIdx.y, threads, tid); c < H && (!MANY || t < p.T); c += threads * gridDim.y * P::N) {
    float acc[P::N];
#pragma unroll
    for (int i = 0; i < P::N; ++i) acc[i] = 0.0f;
    if constexpr (KDOT > 0) {
      P a;
      a.load(v + c, threads, H - c);
      // 4 rows at once, past L2 so that x and dx keep their place in it
      // (fp16, 2051 tokens of 2048, top-8: 16.5 us; 8 at once 17.7, loads kept
      // in L2 29.7).
#pragma unroll
      for (int j0 = 0; j0 < KDOT; j0 += 4) {
        if (j0 >= k) break;
        P b[4];
#pragma unroll
        for (int j = 0; j < 4; ++j)
          if (j0 + j < k && s.row[j0 + j] >= 0) b[j].load_once(rows + (size_t)s.row[j0 + j] * H + c, threads, H - c);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          if (j0 + j >= k || s.row[j0 + j] < 0) continue;
          const float g = s.g[j0 + j];
#pragma unroll
          for (int i = 0; i < P::N; ++i) {
            acc[i] = fmaf(g, b[j].f(i), acc[i]);
            dot[j0 + j] = fmaf(a.f(i), b[j].f(i), dot[j0 + j]);
          }
        }
      }
    } else {
      // 8 rows at once, their loads before their sums (a loop that leaves it to
      // the compiler had one or two in flight: 80 against 69 us at 4096 tokens
      // of 6144, top-8).
#pragma unroll 1
      for (int j0 = 0; j0 < k; j0 += 8) {
        P b[8];
#pragma unroll
        for (int j = 0; j < 8; ++j)
          if (j0 + j < k && s.row[j0 + j] >= 0) b[j].load(rows + (size_t)s.row[j0 + j] * H + c, threads, H - c);
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          if (j0 + j >= k || s.row[j0 + j] < 0) continue;
          const float g = s.g[j0 + j];
#pragma unroll
          for (int i = 0; i < P::N; ++i) acc[i] = fmaf(g, b[j].f(i), acc[i]);
        }
      }
    }
    P o;
#pragma unroll
    for (int i = 0; i < P::N; ++i) o.set(i, acc[i]);
    o.store(out + c, threads, H - c);
  }
  if constexpr (KDOT > 0) token_dots<KDOT>(p, t, dot, s_dots, s);
}

// ------------------------------------------------------------ launchers
static bool rows_vectorised(const RowsParams& p) {
  const int es = p.row_dtype == ROW_F32 ? 4 : 2;
  const uintptr_t all = (uintptr_t)p.v | (uintptr_t)p.other | (uintptr_t)p.rows_out | (uintptr_t)p.rows_in |
                        (uintptr_t)p.out;
  return ((size_t)p.H * es) % 16 == 0 && all % 16 == 0;
}

// Pieces of a row.
static int pieces(const RowsParams& p, bool vec) {
  const int n = vec && p.row_dtype != ROW_F32 ? 8 : 4;
  return (p.H + n - 1) / n;
}

// Column parts of a token, one load a thread: none of a CTA's time is a second
// round of latency, and small batches reach more SMs (8 tokens of 6144 16-bit
// columns: 24 CTAs). One part where dot products need the whole token.
static unsigned column_parts(const RowsParams& p, bool vec) {
  const int parts = (pieces(p, vec) + ROWS_THREADS - 1) / ROWS_THREADS;
  return (unsigned)(parts < 1 ? 1 : (parts < 65535 ? parts : 65535));
}

// Threads of a token and tokens of a CTA. Where tokens are many and rows narrow,
// a CTA of 256 threads for each costs more than its rows: its start, the slots'
// look-up and the dot products' barriers. So below 256 pieces a token gets as few
// threads as leave each up to 4 pieces, and one piece where rows are only written
// (8192 tokens of 256 16-bit columns, top-8, with 32 threads and with 256:
// dispatch 9.3 and 12.8 us, combine 9.2 and 28.2, their gradients 13.2 and 39.7,
// 16.4 and 47.2; 4096 of 1536, top-4, with 64 and 256: the gradients 15.9 and
// 22.0, 23.8 and 30.7). With 256 pieces and more a token has all threads (2051 of
// 2048, top-8: dispatch's gradient 15.5 us, 17.8 with 128), and so it has where
// tokens are few (300 of 1000: combine 2.1 us, 4.1 with 32).
static dim3 token_block(const RowsParams& p, bool vec, bool reads, int num_sms) {
  const int cols = pieces(p, vec);
  unsigned threads = ROWS_THREADS;
  if (p.T >= 4 * num_sms && cols < ROWS_THREADS)
    while (threads > 32 && cols <= (int)threads / 2 * (reads ? 4 : 1)) threads /= 2;
  return dim3(threads, ROWS_THREADS / threads);
}

template <int DT, bool VEC, bool MANY>
static cudaError_t spread_with(const RowsParams& p, dim3 grid, dim3 block, cudaStream_t st) {
  if (!p.other) return launch_pdl(spread_kernel<DT, VEC, 0, MANY>, grid, block, 0, st, p);
  return p.topk <= 8 ? launch_pdl(spread_kernel<DT, VEC, 8, MANY>, grid, block, 0, st, p)
                     : launch_pdl(spread_kernel<DT, VEC, MAX_TOPK, MANY>, grid, block, 0, st, p);
}
template <int DT, bool VEC>
static cudaError_t spread_as(const RowsParams& p, dim3 grid, dim3 block, cudaStream_t st) {
  return block.y > 1 ? spread_with<DT, VEC, true>(p, grid, block, st) : spread_with<DT, VEC, false>(p, grid, block, st);
}
cudaError_t launch_spread(const RowsParams& p, int num_sms, cudaStream_t st) {
  const bool vec = rows_vectorised(p);
  const int pads = p.has_pads ? (p.R / 8 + 1 < num_sms * 4 ? p.R / 8 + 1 : num_sms * 4) : 0;
  if (p.T == 0) return cudaSuccess;
  const dim3 block = token_block(p, vec, p.other != nullptr, num_sms);
  const dim3 grid(((unsigned)p.T + block.y - 1) / block.y + (unsigned)pads, p.other || block.y > 1 ? 1 : column_parts(p, vec));
  cudaError_t e;
  if (p.row_dtype == ROW_BF16) e = vec ? spread_as<ROW_BF16, true>(p, grid, block, st) : spread_as<ROW_BF16, false>(p, grid, block, st);
  else if (p.row_dtype == ROW_F16) e = vec ? spread_as<ROW_F16, true>(p, grid, block, st) : spread_as<ROW_F16, false>(p, grid, block, st);
  else e = vec ? spread_as<ROW_F32, true>(p, grid, block, st) : spread_as<ROW_F32, false>(p, grid, block, st);
  count_launches(1);
  return e;
}

// At most this many rows go with their plan in one launch: 8 tokens of 6144
// columns, top-8, took 3.9 us in two.
constexpr int DISPATCH_SMALL_ROWS = 1024;
template <int DT, bool VEC>
static cudaError_t small_as(const DispatchPlan& d, const RowsParams& p, unsigned grid, cudaStream_t st) {
  return launch_pdl(dispatch_small_kernel<DT, VEC>, dim3(grid), dim3(MAX_E), 0, st, d, p);
}
cudaError_t launch_dispatch(const RowsParams& p, const int* perm, const int* offsets, int align, int capacity,
                            int* row_slot, int* slot_row, int* row_offsets, int num_sms, cudaStream_t st) {
  const DispatchPlan d{perm, offsets, p.T * p.topk, p.E, align, capacity, p.R, row_slot, slot_row, row_offsets, p.status};
  const int most = p.R > d.S ? p.R : d.S;
  cudaError_t e;
  if (most <= DISPATCH_SMALL_ROWS) {
    const bool vec = rows_vectorised(p);
    const unsigned grid = (unsigned)(p.R < 1 ? 1 : (p.R < 2 * num_sms ? p.R : 2 * num_sms));
    if (p.row_dtype == ROW_BF16) e = vec ? small_as<ROW_BF16, true>(d, p, grid, st) : small_as<ROW_BF16, false>(d, p, grid, st);
    else if (p.row_dtype == ROW_F16) e = vec ? small_as<ROW_F16, true>(d, p, grid, st) : small_as<ROW_F16, false>(d, p, grid, st);
    else e = vec ? small_as<ROW_F32, true>(d, p, grid, st) : small_as<ROW_F32, false>(d, p, grid, st);
    count_launches(1);
    return e;
  }
  const unsigned blocks = ((unsigned)most + MAX_E - 1) / MAX_E, sms = (unsigned)num_sms;
  e = launch_pdl(dispatch_plan_kernel, dim3(blocks < sms ? blocks : sms), dim3(MAX_E), 0, st, d);
  count_launches(1);
  return e == cudaSuccess ? launch_spread(p, num_sms, st) : e;
}

template <int DT, bool VEC, bool MANY>
static cudaError_t collect_with(const RowsParams& p, dim3 grid, dim3 block, cudaStream_t st) {
  if (!p.v) return launch_pdl(collect_kernel<DT, VEC, 0, MANY>, grid, block, 0, st, p);
  return p.topk <= 8 ? launch_pdl(collect_kernel<DT, VEC, 8, MANY>, grid, block, 0, st, p)
                     : launch_pdl(collect_kernel<DT, VEC, MAX_TOPK, MANY>, grid, block, 0, st, p);
}
template <int DT, bool VEC>
static cudaError_t collect_as(const RowsParams& p, dim3 grid, dim3 block, cudaStream_t st) {
  return block.y > 1 ? collect_with<DT, VEC, true>(p, grid, block, st) : collect_with<DT, VEC, false>(p, grid, block, st);
}
cudaError_t launch_collect(const RowsParams& p, int num_sms, cudaStream_t st) {
  if (p.T == 0) return cudaSuccess;
  const bool vec = rows_vectorised(p);
  // Large batches have CTAs enough, and the slots' look-up is paid once a token
  // (4096 tokens of 6144 columns, top-8: 69.3 against 73.3 us).
  const dim3 block = token_block(p, vec, true, num_sms);
  const dim3 grid(((unsigned)p.T + block.y - 1) / block.y, p.v || p.T >= 4 * num_sms ? 1 : column_parts(p, vec));
  cudaError_t e;
  if (p.row_dtype == ROW_BF16) e = vec ? collect_as<ROW_BF16, true>(p, grid, block, st) : collect_as<ROW_BF16, false>(p, grid, block, st);
  else if (p.row_dtype == ROW_F16) e = vec ? collect_as<ROW_F16, true>(p, grid, block, st) : collect_as<ROW_F16, false>(p, grid, block, st);
  else e = vec ? collect_as<ROW_F32, true>(p, grid, block, st) : collect_as<ROW_F32, false>(p, grid, block, st);
  count_launches(1);
  return e;
}

}  // namespace hmoe
