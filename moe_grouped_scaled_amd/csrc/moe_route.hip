// Routing around the expert MLP for gfx950: the top-k experts of every token with their weights, tokens
// sorted by expert and copied into expert order, expert outputs summed back per token, and the gradients
// of all of them.  Entry points, host validation and kernels.
//
// The expert MLP takes rows sorted by expert and their split sizes (page "Activation + GroupedLinear
// Fusion for MOE", sequence diagram); these calls make both from a router's logits and undo the order
// afterwards, with the split sizes left in device memory, so a captured graph follows the routing.
//
// A slot is one (token, choice) pair, numbered token * topk + choice.
#include <algorithm>
#include <cmath>
#include <initializer_list>
#include <type_traits>

#include "mgs_device.h"

namespace mgs {
namespace {

// ------------------------------------------------------------------------------------------ router
//
// Sixteen lanes (one DPP row) own a token, four tokens a wave; lane l holds the logits of experts
// l, l + 16, ... as 32-bit keys that order like the values, the last byte of a key replaced by 255 - expert,
// so that keys are unique and equal values order by expert.  A pick is a maximum over the lane's keys and
// four DPP steps; the next one is the largest key below it: with unsigned wrap-around, key - M is larger
// the closer the key lies below M, and small for the keys already taken, so M + max(key - M) is the next
// pick and nothing has to be marked as taken.  Replacing the last byte is exact for BF16 logits (and FP32
// ones whose last byte is zero); for others a wave in which two neighbouring picks, or the last pick and
// the next key, agree in the other 24 bits picks again with whole keys.
//
// Bound by the picks (VALU): 65536 tokens x 256 FP32 experts, top 8, takes 23 us for 67 MB of logits (13 us at
// the rate of a large copy): 678 VALU instructions a wave, whose issue fills the cycles that a CU is busy (counted).
// 16 tokens x 32 experts 2.0 us, the shortest a launch is here.
constexpr int ROUTE_LANES = 16;
constexpr int DPP_ROW_ROR1 = 0x121, DPP_ROW_ROR2 = 0x122;

__device__ __forceinline__ uint32_t row_umax(uint32_t v) {
  v = umax(v, dpp_u<DPP_ROW_ROR8>(v));
  v = umax(v, dpp_u<DPP_ROW_ROR4>(v));
  v = umax(v, dpp_u<DPP_ROW_ROR2>(v));
  return umax(v, dpp_u<DPP_ROW_ROR1>(v));
}
__device__ __forceinline__ float row_sum(float v) {
  v += dpp_f<DPP_ROW_ROR8>(v);
  v += dpp_f<DPP_ROW_ROR4>(v);
  v += dpp_f<DPP_ROW_ROR2>(v);
  return v + dpp_f<DPP_ROW_ROR1>(v);
}

// Integer that orders like the logit: -0 equals +0 (the addition), NaN above everything.
__device__ __forceinline__ uint32_t logit_key(float x) {
  if (x != x) return 0xffffffffu;
  const uint32_t b = __float_as_uint(x + 0.0f);
  return b & 0x80000000u ? ~b : b | 0x80000000u;
}
__device__ __forceinline__ float key_logit(uint32_t k) {
  return k == 0xffffffffu ? __uint_as_float(0x7fc00000u) : __uint_as_float(k & 0x80000000u ? k ^ 0x80000000u : ~k);
}
constexpr uint32_t KEY_NEG_INF = 0x007fffffu;  // key of -inf; experts that cannot be picked are at or below it

template <typename T>
__device__ __forceinline__ float load_logit(const T* p);
template <>
__device__ __forceinline__ float load_logit<float>(const float* p) { return *p; }
template <>
__device__ __forceinline__ float load_logit<uint16_t>(const uint16_t* p) { return bf16lo(*p); }
__device__ __forceinline__ void store_value(float* p, float v) { *p = v; }
__device__ __forceinline__ void store_value(uint16_t* p, float v) { *p = (uint16_t)bf16x2(v, 0.0f); }

struct RouteArgs {
  int64_t tokens;
  int experts, topk, score, renormalize;
  float scale;
  int64_t ld, ldd;
};

// The topk picks of a token by whole keys: lane c < topk gets choice c (-1: none).  Two reductions and a
// pass that clears the pick, each round.
template <int EPL>
__device__ __forceinline__ int pick_exact(const float (&x)[EPL], int experts, int topk, int l) {
  uint32_t key[EPL];
#pragma unroll
  for (int j = 0; j < EPL; ++j) key[j] = ROUTE_LANES * j + l < experts ? logit_key(x[j]) : 0u;
  int pick = -1;
  for (int c = 0; c < topk; ++c) {
    uint32_t m = key[0];
#pragma unroll
    for (int j = 1; j < EPL; ++j) m = umax(m, key[j]);
    m = row_umax(m);
    int at = -1;
#pragma unroll
    for (int j = EPL - 1; j >= 0; --j) at = key[j] == m ? ROUTE_LANES * j + l : at;
    // lowest expert among the lanes that hold m, as a maximum of the complement
    const int e = (int)~row_umax(at < 0 ? 0u : ~(uint32_t)at);
    if (l == c) pick = m > KEY_NEG_INF ? e : -1;
#pragma unroll
    for (int j = 0; j < EPL; ++j) key[j] = ROUTE_LANES * j + l == e ? 0u : key[j];
  }
  return pick;
}

template <typename T, int EPL>
__global__ __launch_bounds__(256) void route_kernel(RouteArgs a, const T* __restrict__ logits,
                                                    int32_t* __restrict__ idx, float* __restrict__ weights) {
  const int l = threadIdx.x & (ROUTE_LANES - 1);
  const int64_t t = (int64_t)blockIdx.x * (256 / ROUTE_LANES) + (threadIdx.x >> 4);
  const bool there = t < a.tokens;
  const T* row = logits + (there ? t : 0) * a.ld;
  float x[EPL];
#pragma unroll
  for (int j = 0; j < EPL; ++j) {
    const int e = ROUTE_LANES * j + l;
    x[j] = there && e < a.experts ? load_logit(row + e) : -INFINITY;
  }
  uint32_t key[EPL], low = 0;
#pragma unroll
  for (int j = 0; j < EPL; ++j) {
    const int e = ROUTE_LANES * j + l;
    low |= __float_as_uint(x[j]);
    key[j] = e < a.experts ? (logit_key(x[j]) & ~0xffu) | (uint32_t)(255 - e) : 0u;
  }
  // experts at or below this key are not available (-inf with any last byte)
  constexpr uint32_t NONE = KEY_NEG_INF | 0xffu;
  uint32_t m = 0;
#pragma unroll
  for (int j = 0; j < EPL; ++j) m = umax(m, key[j]);
  m = row_umax(m);
  int pick = -1;
  bool again = false;
  for (int c = 0; c < a.topk; ++c) {
    if (l == c && m > NONE) pick = 255 - (int)(m & 0xffu);
    uint32_t d = 0;
#pragma unroll
    for (int j = 0; j < EPL; ++j) d = umax(d, key[j] - m);
    const uint32_t next = m + row_umax(d);
    // next >= m: nothing is left below m
    again |= next < m && next > NONE && ((next ^ m) >> 8) == 0u;
    m = next < m ? next : 0u;
  }
  if (sizeof(T) == 4 && __ballot(again) != 0 && __ballot((low & 0xffu) != 0) != 0) pick = pick_exact<EPL>(x, a.experts, a.topk, l);
  const float v = there && pick >= 0 ? load_logit(row + pick) : 0.0f;
  float p = 0.0f, sum = 0.0f;
  const bool full_sum = a.score == MGS_SCORE_SOFTMAX && !a.renormalize;
  if (a.score == MGS_SCORE_SOFTMAX) {
    const float top = __shfl(v, 0, ROUTE_LANES);  // the first pick is the maximum
    if (pick >= 0) p = expf(v - top);
    if (full_sum) {
#pragma unroll
      for (int j = 0; j < EPL; ++j) sum += x[j] == -INFINITY ? 0.0f : expf(x[j] - top);
      sum = row_sum(sum);
    }
  } else if (pick >= 0) {
    const float z = expf(-fabsf(v));  // in (0, 1]: neither form below overflows
    p = (v >= 0.0f ? 1.0f : z) / (1.0f + z);
  }
  if (a.renormalize) sum = row_sum(p);
  if (there && l < a.topk) {
    idx[t * a.topk + l] = pick;
    float w = p;
    // a sum of 0 (sigmoid scores that all underflow) leaves the weights 0
    if (pick >= 0 && (full_sum || a.renormalize) && sum != 0.0f) w = p / sum;
    weights[t * a.topk + l] = w * a.scale;
  }
}

// Gradient of the weights with respect to the logits.  Lane c of a token's sixteen holds choice c.  The
// differences g_j - sum_i w_i g_i of the softmax and of the renormalization cancel where one weight is
// near 1, so they are taken as sum_i w_i (g_j - g_i), plus g_j times the weight of the experts not picked.
// Bound by bytes: 21 us at 65536 x 256, top 8, renormalized sigmoid (67 MB written, 6 MB of picks and gradients, and
// a 64-byte piece of the logits per pick).
template <typename T, int EPL>
__global__ __launch_bounds__(256) void route_bwd_kernel(RouteArgs a, const T* __restrict__ logits,
                                                        const int32_t* __restrict__ idx,
                                                        const float* __restrict__ dweights,
                                                        T* __restrict__ dlogits) {
  // the token's gradients, laid out by expert, and one slot for choices without one
  __shared__ float out_lds[256 / ROUTE_LANES][ROUTE_LANES * EPL + 1];
  const int l = threadIdx.x & (ROUTE_LANES - 1);
  const int64_t t = (int64_t)blockIdx.x * (256 / ROUTE_LANES) + (threadIdx.x >> 4);
  const bool there = t < a.tokens;
  float* line = out_lds[threadIdx.x >> 4];
  int e = -1;
  float g = 0.0f, x = 0.0f;
  if (there && l < a.topk) {
    e = idx[t * a.topk + l];
    if (e < 0 || e >= a.experts) e = -1;
    if (e >= 0) {
      g = dweights[t * a.topk + l] * a.scale;
      x = load_logit(logits + t * a.ld + e);
    }
  }
  const bool softmax = a.score == MGS_SCORE_SOFTMAX, dense = softmax && !a.renormalize;
  float p = 0.0f, q = 0.0f;  // the choice's score; 1 - score of a sigmoid
  float ex[EPL];
  float rest = 0.0f;         // softmax weight of the experts that were not picked
  if (softmax) {
    // maximum and sum over the picked experts, or over all of them
    const uint32_t best = row_umax(e >= 0 ? logit_key(x) : 0u);
    const float top = best > KEY_NEG_INF ? key_logit(best) : 0.0f;
    float sum;
    p = e >= 0 ? expf(x - top) : 0.0f;
    if (dense) {
      // the picked experts are marked so that the others' sum can be taken on its own
#pragma unroll
      for (int j = 0; j < EPL; ++j) line[ROUTE_LANES * j + l] = 0.0f;
      __builtin_amdgcn_wave_barrier();
      line[e >= 0 ? e : ROUTE_LANES * EPL] = 1.0f;
      __builtin_amdgcn_wave_barrier();
      float s = 0.0f;
#pragma unroll
      for (int j = 0; j < EPL; ++j) {
        const int at = ROUTE_LANES * j + l;
        const bool in = there && at < a.experts;
        ex[j] = in ? expf(load_logit(logits + t * a.ld + at) - top) : 0.0f;
        s += line[at] != 0.0f ? 0.0f : ex[j];
      }
      rest = row_sum(s);
      sum = rest + row_sum(p);
      const float div = sum != 0.0f ? sum : 1.0f;  // 0: no expert is available
      rest /= div;
#pragma unroll
      for (int j = 0; j < EPL; ++j) ex[j] /= div;
    } else {
      sum = row_sum(p);
    }
    p = e >= 0 ? p / sum : 0.0f;
  } else if (e >= 0) {
    const float z = expf(-fabsf(x));  // in (0, 1]: neither form below overflows
    p = (x >= 0.0f ? 1.0f : z) / (1.0f + z);
    q = (x >= 0.0f ? z : 1.0f) / (1.0f + z);
  }
  float w = p;
  if (!softmax && a.renormalize) {
    const float s = row_sum(p);
    w = e >= 0 && s != 0.0f ? p / s : 0.0f;
  }
  float d;
  if (dense || a.renormalize) {
    float s = 0.0f;
    for (int i = 0; i < a.topk; ++i) {
      const float wi = __shfl(w, i, ROUTE_LANES), gi = __shfl(g, i, ROUTE_LANES);
      s = __builtin_fmaf(wi, g - gi, s);
    }
    d = w * __builtin_fmaf(g, rest, s);
    if (!softmax) d *= q;
  } else {
    d = g * p * q;
  }
  const float others = dense ? -row_sum(w * g) : 0.0f;  // of the experts not picked: -p_e sum_i w_i g_i
  __builtin_amdgcn_wave_barrier();
#pragma unroll
  for (int j = 0; j < EPL; ++j) line[ROUTE_LANES * j + l] = dense ? ex[j] * others : 0.0f;
  __builtin_amdgcn_wave_barrier();
  line[e >= 0 ? e : ROUTE_LANES * EPL] = d;
  __builtin_amdgcn_wave_barrier();
#pragma unroll
  for (int j = 0; j < EPL; ++j) {
    const int at = ROUTE_LANES * j + l;
    if (there && at < a.experts) store_value(dlogits + t * a.ldd + at, line[at]);
  }
}

// ------------------------------------------------------------------------------------------ sorting
//
// A stable counting sort of the slots by expert: row_of_slot[s] is the number of slots with a smaller
// expert plus those with the same expert and a smaller number; slots without an expert get -1.  The
// result is fixed by the indices alone.  Two launches of 4.7 and 5.0 us at 32768 slots.

// Slots per histogram block: at most SORT_BLOCKS blocks up to 524288 slots, so that a block's sum over the blocks before
// it stays short.  Beyond that every block would read the counts of all (a square of the slots: 4096 blocks x 4 MB at
// 16.8 M slots and 256 experts), and a launch between the two turns the counts into sums once.  256 experts, replayed
// from a graph: 524288 slots 17.4 us in two launches, 524296 15.0 in three; 8.4 M 45 us, 67 M 273 us.
__host__ __device__ inline int sort_chunk(int64_t slots) { return slots <= 131072 ? 1024 : 4096; }
constexpr int64_t SORT_BLOCKS = 128;

// Up to this many slots the dispatch is one launch whose workgroups each look at all of them.  Replayed from a
// graph, 4096 wide: 8 tokens x top 2 3.0 us (6.8 in the three launches of the general form), 64 x 4 4.3 (7.8),
// 512 x 4 9.2 (10.6), 256 x 8 12.4 (11.5, but two launches more to enqueue).
constexpr int64_t SMALL_SLOTS = 2048;

__device__ __forceinline__ int slot_expert(const int32_t* __restrict__ idx, int64_t s, int64_t slots, int experts) {
  const int e = s < slots ? idx[s] : -1;
  return e >= 0 && e < experts ? e : -1;
}

template <int CHUNK>
__global__ __launch_bounds__(256) void sort_count_kernel(int64_t slots, int experts, const int32_t* __restrict__ idx,
                                                         int32_t* __restrict__ counts) {
  __shared__ int32_t h[MGS_MAX_GROUPS];
  h[threadIdx.x] = 0;
  const int64_t s0 = (int64_t)blockIdx.x * CHUNK;
  int e[CHUNK / 256];
#pragma unroll
  for (int i = 0; i < CHUNK / 256; ++i) e[i] = slot_expert(idx, s0 + 256 * i + threadIdx.x, slots, experts);
  __syncthreads();
#pragma unroll
  for (int i = 0; i < CHUNK / 256; ++i)
    if (e[i] >= 0) atomicAdd(&h[e[i]], 1);
  __syncthreads();
  if ((int)threadIdx.x < experts) counts[(int64_t)blockIdx.x * experts + threadIdx.x] = h[threadIdx.x];
}

// Exclusive sum over the 256 threads of a workgroup.
__device__ __forceinline__ int block_exclusive(int v, int32_t* lds) {
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  int s = v;
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) {
    const int o = __shfl_up(s, d);
    s += lane >= d ? o : 0;
  }
  if (lane == 63) lds[wave] = s;
  __syncthreads();
#pragma unroll
  for (int w = 0; w < 3; ++w) s += w < wave ? lds[w] : 0;
  return s - v;
}

// The counts [blocks x experts] replaced, per expert, by the sums of the blocks before; their totals in one row more.
// A workgroup has 16 experts (whole 64-byte pieces of the rows) and splits the blocks into 64 runs of consecutive ones.
constexpr int SCAN_RUNS = 64;
__global__ __launch_bounds__(1024) void sort_scan_kernel(int blocks, int experts, int32_t* __restrict__ counts) {
  __shared__ int32_t part[SCAN_RUNS][16];
  const int l = threadIdx.x & 15, run = threadIdx.x >> 4, e = 16 * blockIdx.x + l;
  const int per = (blocks + SCAN_RUNS - 1) / SCAN_RUNS;
  const int b0 = min(run * per, blocks), b1 = e < experts ? min(b0 + per, blocks) : b0;
  int32_t* at = counts + (int64_t)b0 * experts + e;
  int sum = 0;
#pragma unroll 8
  for (int i = 0; i < b1 - b0; ++i) sum += at[(int64_t)i * experts];
  part[run][l] = sum;
  __syncthreads();
  int before = 0;
  for (int r = 0; r < run; ++r) before += part[r][l];
#pragma unroll 8
  for (int i = 0; i < b1 - b0; ++i) {
    const int v = at[(int64_t)i * experts];
    at[(int64_t)i * experts] = before;
    before += v;
  }
  if (run == SCAN_RUNS - 1 && e < experts) counts[(int64_t)blocks * experts + e] = before;
}

// SCANNED: the counts are sort_scan_kernel's sums.
template <int CHUNK, bool SCANNED>
__global__ __launch_bounds__(256) void sort_rows_kernel(int64_t slots, int experts, const int32_t* __restrict__ idx,
                                                        const int32_t* __restrict__ counts,
                                                        int32_t* __restrict__ row_of_slot,
                                                        int64_t* __restrict__ splits) {
  __shared__ int32_t scan[4];
  __shared__ int32_t next[4][MGS_MAX_GROUPS];  // the next row of each expert, per wave
  const int t = threadIdx.x, lane = t & 63, wave = t >> 6;
  // wave w owns the w-th quarter of the chunk; its rows follow those of the waves before it
  constexpr int PER = CHUNK / 4;
  const int64_t s0 = (int64_t)blockIdx.x * CHUNK + (int64_t)wave * PER;
  int e[PER / 64];
#pragma unroll
  for (int i = 0; i < PER / 64; ++i) e[i] = slot_expert(idx, s0 + 64 * i + lane, slots, experts);
  int before = 0, total = 0;
  if (t < experts) {
    const int nb = gridDim.x;
    if constexpr (SCANNED) {
      before = counts[(int64_t)blockIdx.x * experts + t];
      total = counts[(int64_t)nb * experts + t];
    } else {
#pragma unroll 8
      for (int b = 0; b < nb; ++b) {
        const int v = counts[(int64_t)b * experts + t];
        before += b < (int)blockIdx.x ? v : 0;
        total += v;
      }
    }
    if (blockIdx.x == 0) splits[t] = total;
  }
#pragma unroll
  for (int w = 0; w < 4; ++w) next[w][t] = 0;
  int r = block_exclusive(total, scan) + before;  // (its barrier also stands between the zeros and the counts)
#pragma unroll
  for (int i = 0; i < PER / 64; ++i)
    if (e[i] >= 0) atomicAdd(&next[wave][e[i]], 1);
  __syncthreads();
#pragma unroll
  for (int w = 0; w < 4; ++w) {
    const int c = next[w][t];
    next[w][t] = r;
    r += c;
  }
  __syncthreads();
#pragma unroll
  for (int i = 0; i < PER / 64; ++i) {
    const int64_t s = s0 + 64 * i + lane;
    // lanes with the same expert: one ballot per bit of it
    uint64_t same = __ballot(e[i] >= 0);
#pragma unroll
    for (int b = 0; b < 8; ++b) {
      const uint64_t v = __ballot((e[i] >> b) & 1);
      same &= (e[i] >> b) & 1 ? v : ~v;
    }
    const int rank = __popcll(same & ((1ull << lane) - 1));
    int row = -1;
    if (e[i] >= 0) row = next[wave][e[i]] + rank;
    __builtin_amdgcn_wave_barrier();
    if (e[i] >= 0 && rank == 0) next[wave][e[i]] += __popcll(same);
    __builtin_amdgcn_wave_barrier();
    if (s < slots) row_of_slot[s] = row;
  }
}

// ------------------------------------------------------------------------------------------ row copies
//
// Rows are moved in units of V elements (16 bytes where widths, strides and addresses allow it, else
// single elements).  A token's units are spread over `tpt` threads, a power of two up to 256.

// the same bits, unconverted
template <typename T, int V>
struct Raw { typedef uint4 type; };
template <>
struct Raw<float, 1> { typedef float type; };
template <>
struct Raw<uint16_t, 1> { typedef uint16_t type; };

template <typename T, int V>
__device__ __forceinline__ void unit_unpack(const typename Raw<T, V>::type& w, float (&v)[V]) {
  if constexpr (V == 8) {
    unpack8(w, v);
  } else if constexpr (V == 4) {
    v[0] = __uint_as_float(w.x); v[1] = __uint_as_float(w.y); v[2] = __uint_as_float(w.z); v[3] = __uint_as_float(w.w);
  } else {
    v[0] = load_logit(&w);
  }
}

template <typename T, int V>
__device__ __forceinline__ void unit_load(const T* p, float (&v)[V]) {
  unit_unpack<T, V>(*reinterpret_cast<const typename Raw<T, V>::type*>(p), v);
}

// The data registers of a 16-byte store stay live through two wait states after it (a VALU write to one of
// them in the next instruction changed what part of the wave stored).
// NT: non-temporal, for tensors far larger than the caches (see streams()).
typedef unsigned int v4u_t __attribute__((ext_vector_type(4)));
template <bool NT>
__device__ __forceinline__ void store16(void* p, uint4 d) {
  const v4u_t v = {d.x, d.y, d.z, d.w};
  if constexpr (NT) __builtin_nontemporal_store(v, reinterpret_cast<v4u_t*>(p));
  else *reinterpret_cast<v4u_t*>(p) = v;
  asm volatile("s_nop 1" ::"v"(v));
}

template <typename T, int V, bool NT>
__device__ __forceinline__ void unit_store(T* p, const float (&v)[V]) {
  if constexpr (V == 8) {
    store16<NT>(p, pack8_bf16(v));
  } else if constexpr (V == 4) {
    store16<NT>(p, make_uint4(__float_as_uint(v[0]), __float_as_uint(v[1]), __float_as_uint(v[2]), __float_as_uint(v[3])));
  } else {
    store_value(p, v[0]);
  }
}

template <bool NT>
__device__ __forceinline__ void raw_store(uint4* p, uint4 v) { store16<NT>(p, v); }
template <bool NT>
__device__ __forceinline__ void raw_store(float* p, float v) { *p = v; }
template <bool NT>
__device__ __forceinline__ void raw_store(uint16_t* p, uint16_t v) { *p = v; }
template <bool NT, typename R>
__device__ __forceinline__ R raw_load(const R* p) {
  if constexpr (NT && sizeof(R) == 16) {
    const v4u_t v = __builtin_nontemporal_load(reinterpret_cast<const v4u_t*>(p));
    return make_uint4(v[0], v[1], v[2], v[3]);
  } else {
    return *p;
  }
}

struct MoveArgs {
  int64_t tokens, hidden, ld;  // ld: row stride of the token-side tensor (elements)
  int topk, experts;
  int32_t num_rows;            // rows of the expert-side tensor
  int tpt_log2;                // threads per token
};

// row of a slot, -1 where it has none
__device__ __forceinline__ int slot_row(const MoveArgs& a, const int32_t* __restrict__ row_of_slot, int64_t t, int c) {
  const int r = row_of_slot[t * a.topk + c];
  return r >= 0 && r < a.num_rows ? r : -1;
}

// x row of every token into the rows of its slots (the token's unit is read once).  Bound by bytes: 74 us for
// 403 MB (16384 tokens x 4096, top 2: 5.4 TB/s, mostly writes).
template <typename T, int V, int KMAX, bool NT>
__device__ __forceinline__ void scatter_row(const MoveArgs& a, const int (&r)[KMAX], const T* __restrict__ x,
                                            T* __restrict__ rows, int u, int tpt) {
  typedef typename Raw<T, V>::type R;
  for (int64_t h = (int64_t)u * V; h < a.hidden; h += (int64_t)V * tpt) {
    const R v = *reinterpret_cast<const R*>(x + h);
#pragma unroll
    for (int c = 0; c < KMAX; ++c)
      if (c < a.topk && r[c] >= 0) raw_store<NT>(reinterpret_cast<R*>(rows + (int64_t)r[c] * a.hidden + h), v);
  }
}

template <typename T, int V, int KMAX, bool NT>
__global__ __launch_bounds__(256) void scatter_kernel(MoveArgs a, const int32_t* __restrict__ row_of_slot,
                                                      const T* __restrict__ x, const float* __restrict__ weights,
                                                      T* __restrict__ rows, float* __restrict__ row_weights) {
  const int tpt = 1 << a.tpt_log2, u = threadIdx.x & (tpt - 1);
  const int64_t t = ((int64_t)blockIdx.x << (8 - a.tpt_log2)) + (threadIdx.x >> a.tpt_log2);
  if (t >= a.tokens) return;
  if (row_weights) {
    for (int c = u; c < a.topk; c += tpt) {
      const int r = slot_row(a, row_of_slot, t, c);
      if (r >= 0) row_weights[r] = weights[t * a.topk + c];
    }
  }
  int r[KMAX];
#pragma unroll
  for (int c = 0; c < KMAX; ++c) r[c] = c < a.topk ? slot_row(a, row_of_slot, t, c) : -1;
  scatter_row<T, V, KMAX, NT>(a, r, x + t * a.ld, rows, u, tpt);
}

// The whole dispatch in one launch, for few slots: a workgroup per token counts, over all slots, those that
// precede each of its own in the sorted order, then copies its row.  Workgroup 0 also takes the split sizes.
template <typename T, int V, int KMAX>
__global__ __launch_bounds__(256) void dispatch_small_kernel(MoveArgs a, int slots, const int32_t* __restrict__ idx,
                                                             const T* __restrict__ x, const float* __restrict__ weights,
                                                             T* __restrict__ rows, float* __restrict__ row_weights,
                                                             int32_t* __restrict__ row_of_slot,
                                                             int64_t* __restrict__ splits) {
  __shared__ int32_t part[4][KMAX];
  __shared__ int32_t hist[MGS_MAX_GROUPS];
  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int64_t t = blockIdx.x;
  const int slot0 = (int)t * a.topk;
  int mine[KMAX], n[KMAX];
#pragma unroll
  for (int c = 0; c < KMAX; ++c) {
    n[c] = 0;
    mine[c] = c < a.topk && t < a.tokens ? slot_expert(idx, slot0 + c, slots, a.experts) : -1;
  }
  hist[tid] = 0;
  __syncthreads();
  for (int s0 = 64 * wave; s0 < slots; s0 += 256) {
    const int s = s0 + lane;
    const int e = slot_expert(idx, s, slots, a.experts);
    if (blockIdx.x == 0 && e >= 0) atomicAdd(&hist[e], 1);
#pragma unroll
    for (int c = 0; c < KMAX; ++c)
      if (c < a.topk) n[c] += __popcll(__ballot(e >= 0 && (e < mine[c] || (e == mine[c] && s < slot0 + c))));
  }
#pragma unroll
  for (int c = 0; c < KMAX; ++c)
    if (lane == c) part[wave][c] = n[c];
  __syncthreads();
  if (blockIdx.x == 0 && tid < a.experts) splits[tid] = hist[tid];
  if (t >= a.tokens) return;
  int r[KMAX];
#pragma unroll
  for (int c = 0; c < KMAX; ++c) {
    r[c] = mine[c] >= 0 ? part[0][c] + part[1][c] + part[2][c] + part[3][c] : -1;
    if (tid == c && c < a.topk) {
      row_of_slot[slot0 + c] = r[c];
      if (row_weights && r[c] >= 0) row_weights[r[c]] = weights[slot0 + c];
    }
  }
  if (rows) scatter_row<T, V, KMAX, false>(a, r, x + t * a.ld, rows, tid, 256);
}

// y of every token: the sum over its slots' rows in slot order, in FP32, with weights if given.  Row numbers
// and weights are read once; the loads of eight rows go out before their sums.  Bound by bytes: 67 us for 403 MB
// (16384 tokens x 4096, top 2: 6.0 TB/s, mostly reads), 195 us for 1.06 GB (8192 x 7168, top 8).
template <typename T, int V, int KMAX, bool NT>
__global__ __launch_bounds__(256) void combine_kernel(MoveArgs a, const int32_t* __restrict__ row_of_slot,
                                                      const T* __restrict__ rows, const float* __restrict__ weights,
                                                      T* __restrict__ y, const float* __restrict__ drow_weights,
                                                      float* __restrict__ dweights) {
  typedef typename Raw<T, V>::type R;
  constexpr int GROUP = KMAX < 8 ? KMAX : 8;
  const int tpt = 1 << a.tpt_log2, u = threadIdx.x & (tpt - 1);
  const int64_t t = ((int64_t)blockIdx.x << (8 - a.tpt_log2)) + (threadIdx.x >> a.tpt_log2);
  if (t >= a.tokens) return;
  if (dweights) {
    for (int c = u; c < a.topk; c += tpt) {
      const int r = slot_row(a, row_of_slot, t, c);
      dweights[t * a.topk + c] = r >= 0 ? drow_weights[r] : 0.0f;
    }
  }
  int r[KMAX];
  float w[KMAX];
#pragma unroll
  for (int c = 0; c < KMAX; ++c) {
    r[c] = c < a.topk ? slot_row(a, row_of_slot, t, c) : -1;
    w[c] = weights && r[c] >= 0 ? weights[t * a.topk + c] : 1.0f;
  }
  for (int64_t h = (int64_t)u * V; h < a.hidden; h += (int64_t)V * tpt) {
    float acc[V];
#pragma unroll
    for (int i = 0; i < V; ++i) acc[i] = 0.0f;
#pragma unroll
    for (int c0 = 0; c0 < KMAX; c0 += GROUP) {
      if (c0 >= a.topk) break;
      R v[GROUP];
#pragma unroll
      for (int c = 0; c < GROUP; ++c)
        if (r[c0 + c] >= 0) v[c] = raw_load<NT>(reinterpret_cast<const R*>(rows + (int64_t)r[c0 + c] * a.hidden + h));
#pragma unroll
      for (int c = 0; c < GROUP; ++c) {
        if (r[c0 + c] < 0) continue;
        float f[V];
        unit_unpack<T, V>(v[c], f);
#pragma unroll
        for (int i = 0; i < V; ++i) acc[i] = __builtin_fmaf(w[c0 + c], f[i], acc[i]);
      }
    }
    unit_store<T, V, NT>(y + t * a.ld + h, acc);
  }
}

// d(rows) = w dy and d(w) = <dy, rows>, four slots of a token at a time: a unit of dy is read once for them.
// The sums run over the token's threads by lane exchanges, then over its waves in order.  Bound by bytes: 114 us for
// 671 MB (16384 tokens x 4096 BF16, top 2: 5.9 TB/s), 369 us for 2.0 GB (8192 x 7168, top 8).  10 us for 1021 tokens x
// 1001 FP32, top 3 (23 MB): single elements, four dependent passes a row; with the passes' loads ahead of their
// sums it took 9.5.
template <typename T, int V, bool NT>
__global__ __launch_bounds__(256) void combine_bwd_kernel(MoveArgs a, const int32_t* __restrict__ row_of_slot,
                                                          const T* __restrict__ dy, const T* __restrict__ rows,
                                                          const float* __restrict__ weights, T* __restrict__ drows,
                                                          float* __restrict__ dweights) {
  __shared__ float part[4][4];
  const int tpt = 1 << a.tpt_log2, u = threadIdx.x & (tpt - 1);
  const int64_t t = ((int64_t)blockIdx.x << (8 - a.tpt_log2)) + (threadIdx.x >> a.tpt_log2);
  const bool there = t < a.tokens;
  const int width = tpt < 64 ? tpt : 64;
  for (int c0 = 0; c0 < a.topk; c0 += 4) {
    int r[4];
    float w[4], dot[4];
#pragma unroll
    for (int c = 0; c < 4; ++c) {
      r[c] = there && c0 + c < a.topk ? slot_row(a, row_of_slot, t, c0 + c) : -1;
      w[c] = r[c] >= 0 && weights ? weights[t * a.topk + c0 + c] : 1.0f;
      dot[c] = 0.0f;
    }
    if (there) {
      for (int64_t h = (int64_t)u * V; h < a.hidden; h += (int64_t)V * tpt) {
        float g[V];
        unit_load<T, V>(dy + t * a.ld + h, g);
        if (dweights) {
          typedef typename Raw<T, V>::type R;
          R v[4];
#pragma unroll
          for (int c = 0; c < 4; ++c)
            if (r[c] >= 0) v[c] = raw_load<NT>(reinterpret_cast<const R*>(rows + (int64_t)r[c] * a.hidden + h));
#pragma unroll
          for (int c = 0; c < 4; ++c)
            if (r[c] >= 0) {
              float f[V];
              unit_unpack<T, V>(v[c], f);
#pragma unroll
              for (int i = 0; i < V; ++i) dot[c] = __builtin_fmaf(g[i], f[i], dot[c]);
            }
        }
        if (drows) {
#pragma unroll
          for (int c = 0; c < 4; ++c) {
            float o[V];
#pragma unroll
            for (int i = 0; i < V; ++i) o[i] = w[c] * g[i];
            if (r[c] >= 0) unit_store<T, V, NT>(drows + (int64_t)r[c] * a.hidden + h, o);
          }
        }
      }
    }
    if (!dweights) continue;
#pragma unroll
    for (int c = 0; c < 4; ++c)
      for (int d = width >> 1; d; d >>= 1) dot[c] += __shfl_xor(dot[c], d);
    if (tpt > 64) {
      __syncthreads();
#pragma unroll
      for (int c = 0; c < 4; ++c)
        if ((threadIdx.x & 63) == 0) part[threadIdx.x >> 6][c] = dot[c];
      __syncthreads();
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        const int w0 = (threadIdx.x >> a.tpt_log2) << (a.tpt_log2 - 6);  // the token's first wave
        dot[c] = part[w0][c] + part[w0 + 1][c];
        if (tpt == 256) dot[c] += part[2][c] + part[3][c];
      }
    }
#pragma unroll
    for (int c = 0; c < 4; ++c)
      if (there && u == 0 && c0 + c < a.topk) dweights[t * a.topk + c0 + c] = r[c] >= 0 ? dot[c] : 0.0f;
  }
}

// ------------------------------------------------------------------------------------------ host side

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

// calls f(element type, elements per unit) for rows of `dtype`
template <typename F>
void with_unit(int dtype, bool wide, F f) {
  if (dtype == MGS_DTYPE_BF16) {
    if (wide) f(uint16_t{}, std::integral_constant<int, 8>{});
    else f(uint16_t{}, std::integral_constant<int, 1>{});
  } else {
    if (wide) f(float{}, std::integral_constant<int, 4>{});
    else f(float{}, std::integral_constant<int, 1>{});
  }
}

// Whether the expert-side rows are far larger than the caches (32 MiB of L2), so that what is read or
// written once should not displace what the caches hold: 268 MB of rows (16384 tokens x 4096, top 2) moved and
// summed in 148 us with non-temporal accesses, 165 us without; 940 MB (8192 x 7168, top 8) 401 and 451 us.
bool streams(int64_t tokens, int topk, int64_t hidden, int dtype) {
  return tokens * topk * hidden * (dtype == MGS_DTYPE_BF16 ? 2 : 4) >= (int64_t)128 << 20;
}
template <typename F>
void with_flag(bool v, F f) {
  if (v) f(std::true_type{});
  else f(std::false_type{});
}

// calls f(bound of topk): per-slot registers are sized by it (two slots in arrays of sixteen cost the combine
// of 16384 tokens x 4096 108 instead of 92 us)
template <typename F>
void with_topk(int topk, F f) {
  if (topk <= 2) f(std::integral_constant<int, 2>{});
  else if (topk <= 4) f(std::integral_constant<int, 4>{});
  else if (topk <= 8) f(std::integral_constant<int, 8>{});
  else f(std::integral_constant<int, 16>{});
}

// A launch has at most 2^32 - 1 threads in a dimension.
int check_blocks(int64_t blocks) {
  if (blocks > UINT32_MAX / 256) return fail(MGS_ERR_SHAPE, "%lld workgroups: too many tokens for one call", (long long)blocks);
  return MGS_OK;
}

// 16-byte units need whole units per row, aligned rows and aligned tensors
bool wide_rows(int dtype, int64_t hidden, int64_t ld, std::initializer_list<const void*> ptrs) {
  const int n = dtype == MGS_DTYPE_BF16 ? 8 : 4;
  if (hidden % n || ld % n) return false;
  for (const void* p : ptrs)
    if (p && !aligned16(p)) return false;
  return true;
}

// Memory of a tensor of a call; of rows with a stride only the first, so that tensors side by side in one buffer
// do not count as overlapping.
struct Span {
  const char* name;
  const void* p;
  int64_t bytes;
};
Span span(const char* name, const void* p, int64_t bytes) { return {name, p, p ? bytes : 0}; }
Span span_rows(const char* name, const void* p, int64_t rows, int64_t width, int64_t ld, int dtype) {
  const int64_t es = dtype == MGS_DTYPE_BF16 ? 2 : 4;
  if (!p) return span(name, p, 0);  // (its width was not checked)
  return span(name, p, (ld == width ? rows : std::min<int64_t>(rows, 1)) * width * es);
}

// No output may overlap another tensor of the call: workgroups read and write in any order.
int check_overlap(std::initializer_list<Span> outs, std::initializer_list<Span> ins) {
  auto meet = [](const Span& a, const Span& b) {
    const uintptr_t x = reinterpret_cast<uintptr_t>(a.p), y = reinterpret_cast<uintptr_t>(b.p);
    return a.bytes > 0 && b.bytes > 0 && (x < y ? y - x < (uintptr_t)a.bytes : x - y < (uintptr_t)b.bytes);
  };
  for (const Span* o = outs.begin(); o != outs.end(); ++o) {
    for (const Span* q = o + 1; q != outs.end(); ++q)
      if (meet(*o, *q)) return fail(MGS_ERR_INVALID_ARG, "%s must not be or overlap %s", o->name, q->name);
    for (const Span& i : ins)
      if (meet(*o, i)) return fail(MGS_ERR_INVALID_ARG, "%s must not be or overlap %s", o->name, i.name);
  }
  return MGS_OK;
}

// Threads per token and the launch's workgroups, for rows moved in 16-byte units or single elements.
int set_grid(MoveArgs* a, int dtype, bool wide, int64_t* blocks) {
  const int64_t v = wide ? (dtype == MGS_DTYPE_BF16 ? 8 : 4) : 1, units = (a->hidden + v - 1) / v;
  a->tpt_log2 = 0;
  while (a->tpt_log2 < 8 && ((int64_t)1 << a->tpt_log2) < units) ++a->tpt_log2;
  const int64_t per = 256 >> a->tpt_log2;
  *blocks = (a->tokens + per - 1) / per;
  return check_blocks(*blocks);
}

int check_route(const mgs_route_params* rp, int64_t tokens, int32_t experts, int32_t topk, const void* logits,
                int32_t dtype, int64_t ld, RouteArgs* a) {
  if (!rp) return fail(MGS_ERR_INVALID_ARG, "route params are NULL");
  if (rp->score != MGS_SCORE_SOFTMAX && rp->score != MGS_SCORE_SIGMOID)
    return fail(MGS_ERR_INVALID_ARG, "unknown score function %d", rp->score);
  if (!std::isfinite(rp->scale)) return fail(MGS_ERR_INVALID_ARG, "scale must be finite");
  if (experts < 1 || experts > MGS_MAX_GROUPS)
    return fail(MGS_ERR_INVALID_ARG, "num_experts %d outside [1, %d]", experts, MGS_MAX_GROUPS);
  if (topk < 1 || topk > MGS_MAX_TOPK || topk > experts)
    return fail(MGS_ERR_INVALID_ARG, "topk %d outside [1, min(%d, num_experts %d)]", topk, MGS_MAX_TOPK, experts);
  if (tokens < 0 || tokens > INT32_MAX / topk) return fail(MGS_ERR_SHAPE, "tokens %lld: tokens x topk must be in [0, 2^31)", (long long)tokens);
  if (dtype != MGS_DTYPE_BF16 && dtype != MGS_DTYPE_F32) return fail(MGS_ERR_INVALID_ARG, "unknown logits dtype %d", dtype);
  if (ld < experts) return fail(MGS_ERR_SHAPE, "row stride %lld below the %d experts", (long long)ld, experts);
  if (!logits && tokens > 0) return fail(MGS_ERR_INVALID_ARG, "logits is NULL");
  *a = RouteArgs{tokens, experts, topk, rp->score, rp->renormalize != 0, rp->scale, ld, 0};
  return MGS_OK;
}

int check_move(int64_t tokens, int32_t topk, int64_t hidden, int32_t dtype, int64_t ld, int64_t num_rows, MoveArgs* a) {
  if (topk < 1 || topk > MGS_MAX_TOPK) return fail(MGS_ERR_INVALID_ARG, "topk %d outside [1, %d]", topk, MGS_MAX_TOPK);
  if (tokens < 0 || tokens > INT32_MAX / topk) return fail(MGS_ERR_SHAPE, "tokens %lld: tokens x topk must be in [0, 2^31)", (long long)tokens);
  if (hidden < 1 || hidden > (int64_t)1 << 24) return fail(MGS_ERR_SHAPE, "hidden %lld outside [1, 2^24]", (long long)hidden);
  if (ld < hidden) return fail(MGS_ERR_SHAPE, "row stride %lld below the width %lld", (long long)ld, (long long)hidden);
  if (dtype != MGS_DTYPE_BF16 && dtype != MGS_DTYPE_F32) return fail(MGS_ERR_INVALID_ARG, "unknown dtype %d", dtype);
  if (num_rows < 0 || num_rows > INT32_MAX) return fail(MGS_ERR_SHAPE, "num_rows %lld outside [0, 2^31)", (long long)num_rows);
  *a = MoveArgs{tokens, hidden, ld, topk, 0, (int32_t)num_rows, 0};
  return MGS_OK;
}

int launched() {
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess) return fail(MGS_ERR_HIP, "HIP launch error: %s", hipGetErrorString(e));
  return ok();
}

template <typename F>
void with_experts(int experts, F f) {
  if (experts <= 16) f(std::integral_constant<int, 1>{});
  else if (experts <= 32) f(std::integral_constant<int, 2>{});
  else if (experts <= 64) f(std::integral_constant<int, 4>{});
  else if (experts <= 128) f(std::integral_constant<int, 8>{});
  else f(std::integral_constant<int, 16>{});
}

}  // namespace
}  // namespace mgs

using namespace mgs;

extern "C" {

int mgs_moe_route(const mgs_route_params* rp, int64_t tokens, int32_t experts, int32_t topk, const void* logits,
                  int32_t logits_dtype, int64_t ld, int32_t* expert_idx, float* weights, void* stream) {
  RouteArgs a;
  int rc = check_route(rp, tokens, experts, topk, logits, logits_dtype, ld, &a);
  if (rc) return rc;
  if ((!expert_idx || !weights) && tokens > 0) return fail(MGS_ERR_INVALID_ARG, "expert_idx or weights is NULL");
  if (tokens == 0) return ok();
  if ((rc = check_blocks((tokens + 15) / 16))) return rc;
  if ((rc = check_overlap({span("expert_idx", expert_idx, tokens * topk * 4), span("weights", weights, tokens * topk * 4)},
                          {span_rows("logits", logits, tokens, experts, ld, logits_dtype)})))
    return rc;
  const dim3 grid((unsigned)((tokens + 15) / 16));
  const hipStream_t st = static_cast<hipStream_t>(stream);
  with_experts(experts, [&](auto n) {
    if (logits_dtype == MGS_DTYPE_BF16)
      hipLaunchKernelGGL((route_kernel<uint16_t, decltype(n)::value>), grid, dim3(256), 0, st, a, static_cast<const uint16_t*>(logits), expert_idx, weights);
    else
      hipLaunchKernelGGL((route_kernel<float, decltype(n)::value>), grid, dim3(256), 0, st, a, static_cast<const float*>(logits), expert_idx, weights);
  });
  return launched();
}

int mgs_moe_route_bwd(const mgs_route_params* rp, int64_t tokens, int32_t experts, int32_t topk, const void* logits,
                      int32_t logits_dtype, int64_t ld, const int32_t* expert_idx, const float* dweights,
                      void* dlogits, int64_t ld_dlogits, void* stream) {
  RouteArgs a;
  int rc = check_route(rp, tokens, experts, topk, logits, logits_dtype, ld, &a);
  if (rc) return rc;
  if (ld_dlogits < experts) return fail(MGS_ERR_SHAPE, "row stride %lld of dlogits below the %d experts", (long long)ld_dlogits, experts);
  if ((!expert_idx || !dweights || !dlogits) && tokens > 0)
    return fail(MGS_ERR_INVALID_ARG, "expert_idx, dweights or dlogits is NULL");
  if (tokens == 0) return ok();
  if ((rc = check_blocks((tokens + 15) / 16))) return rc;
  if ((rc = check_overlap({span_rows("dlogits", dlogits, tokens, experts, ld_dlogits, logits_dtype)},
                          {span_rows("logits", logits, tokens, experts, ld, logits_dtype),
                           span("expert_idx", expert_idx, tokens * topk * 4), span("dweights", dweights, tokens * topk * 4)})))
    return rc;
  a.ldd = ld_dlogits;
  const dim3 grid((unsigned)((tokens + 15) / 16));
  const hipStream_t st = static_cast<hipStream_t>(stream);
  with_experts(experts, [&](auto n) {
    if (logits_dtype == MGS_DTYPE_BF16)
      hipLaunchKernelGGL((route_bwd_kernel<uint16_t, decltype(n)::value>), grid, dim3(256), 0, st, a, static_cast<const uint16_t*>(logits), expert_idx, dweights, static_cast<uint16_t*>(dlogits));
    else
      hipLaunchKernelGGL((route_bwd_kernel<float, decltype(n)::value>), grid, dim3(256), 0, st, a, static_cast<const float*>(logits), expert_idx, dweights, static_cast<float*>(dlogits));
  });
  return launched();
}

int64_t mgs_moe_dispatch_workspace_bytes(int64_t tokens, int32_t topk, int32_t experts) {
  if (topk < 1 || topk > MGS_MAX_TOPK) return fail(MGS_ERR_INVALID_ARG, "topk %d outside [1, %d]", topk, MGS_MAX_TOPK);
  if (experts < 1 || experts > MGS_MAX_GROUPS)
    return fail(MGS_ERR_INVALID_ARG, "num_experts %d outside [1, %d]", experts, MGS_MAX_GROUPS);
  if (tokens < 0 || tokens > INT32_MAX / topk) return fail(MGS_ERR_SHAPE, "tokens %lld: tokens x topk must be in [0, 2^31)", (long long)tokens);
  const int64_t slots = tokens * topk, chunk = sort_chunk(slots), blocks = (slots + chunk - 1) / chunk;
  ok();
  if (slots <= SMALL_SLOTS) return 0;
  return 4 * (blocks + (blocks > SORT_BLOCKS ? 1 : 0)) * experts;
}

int mgs_moe_dispatch(int64_t tokens, int32_t topk, int32_t experts, const int32_t* expert_idx, int64_t hidden,
                     int32_t dtype, const void* x, int64_t ldx, const float* weights, void* rows, int64_t num_rows,
                     float* row_weights, int32_t* row_of_slot, int64_t* split_sizes, void* workspace,
                     int64_t workspace_bytes, void* stream) {
  const int64_t need = mgs_moe_dispatch_workspace_bytes(tokens, topk, experts);
  if (need < 0) return (int)need;
  MoveArgs a{};
  int rc;
  const int64_t slots = tokens * topk;
  if (x || rows || weights || row_weights) {
    if ((rc = check_move(tokens, topk, hidden, dtype, ldx, num_rows, &a))) return rc;
    if ((!x || !rows) && tokens > 0) return fail(MGS_ERR_INVALID_ARG, "x and rows go together");
    if (tokens > 0 && (weights == nullptr) != (row_weights == nullptr))
      return fail(MGS_ERR_INVALID_ARG, "weights and row_weights go together");
    if (num_rows < slots)
      return fail(MGS_ERR_SHAPE, "rows has %lld rows, %lld tokens x topk %d can need %lld", (long long)num_rows, (long long)tokens, topk, (long long)slots);
  }
  if (!expert_idx && tokens > 0) return fail(MGS_ERR_INVALID_ARG, "expert_idx is NULL");
  if (!row_of_slot && tokens > 0) return fail(MGS_ERR_INVALID_ARG, "row_of_slot is NULL");
  if (!split_sizes) return fail(MGS_ERR_INVALID_ARG, "split_sizes is NULL");
  if (need > 0 && (!workspace || workspace_bytes < need))
    return fail(MGS_ERR_INVALID_ARG, "the sort needs a workspace of %lld bytes (got %lld%s)", (long long)need,
                (long long)workspace_bytes, workspace ? "" : ", NULL");
  const bool wide = x && wide_rows(dtype, hidden, ldx, {x, rows});
  int64_t blocks = 0;
  if (x && (rc = set_grid(&a, dtype, wide, &blocks))) return rc;
  // (rows past the slots are not written)
  if ((rc = check_overlap({span("row_of_slot", row_of_slot, slots * 4), span("split_sizes", split_sizes, experts * (int64_t)8),
                           span_rows("rows", rows, slots, hidden, hidden, dtype), span("row_weights", row_weights, slots * 4),
                           span("the workspace", workspace, need)},
                          {span("expert_idx", expert_idx, slots * 4), span_rows("x", x, tokens, hidden, ldx, dtype),
                           span("weights", weights, slots * 4)})))
    return rc;
  const hipStream_t st = static_cast<hipStream_t>(stream);
  a.experts = experts;
  a.topk = topk;
  a.tokens = tokens;
  if (slots <= SMALL_SLOTS) {
    with_unit(dtype, wide, [&](auto e, auto n) {
      typedef decltype(e) T;
      with_topk(topk, [&](auto k) {
        hipLaunchKernelGGL((dispatch_small_kernel<T, decltype(n)::value, decltype(k)::value>), dim3((unsigned)std::max<int64_t>(1, tokens)),
                           dim3(256), 0, st, a, (int)slots, expert_idx, static_cast<const T*>(x), weights,
                           static_cast<T*>(tokens ? rows : nullptr), row_weights, row_of_slot, split_sizes);
      });
    });
    return launched();
  }
  int32_t* counts = static_cast<int32_t*>(workspace);
  auto sort = [&](auto c, auto scanned) {
    constexpr int CHUNK = decltype(c)::value;
    constexpr bool SCANNED = decltype(scanned)::value;
    const dim3 grid((unsigned)((slots + CHUNK - 1) / CHUNK));
    hipLaunchKernelGGL(sort_count_kernel<CHUNK>, grid, dim3(256), 0, st, slots, experts, expert_idx, counts);
    if (SCANNED)
      hipLaunchKernelGGL(sort_scan_kernel, dim3((unsigned)((experts + 15) / 16)), dim3(1024), 0, st, (int)grid.x, experts, counts);
    hipLaunchKernelGGL((sort_rows_kernel<CHUNK, SCANNED>), grid, dim3(256), 0, st, slots, experts, expert_idx, counts, row_of_slot, split_sizes);
  };
  // (chunks of 1024 slots: at most 128 blocks)
  if (sort_chunk(slots) == 1024) sort(std::integral_constant<int, 1024>{}, std::false_type{});
  else if (slots <= SORT_BLOCKS * 4096) sort(std::integral_constant<int, 4096>{}, std::false_type{});
  else sort(std::integral_constant<int, 4096>{}, std::true_type{});
  if (x) {
    with_unit(dtype, wide, [&](auto e, auto n) {
      typedef decltype(e) T;
      constexpr int V = decltype(n)::value;
      with_flag(V > 1 && streams(tokens, topk, hidden, dtype), [&](auto nt) {
        with_topk(topk, [&](auto k) {
          hipLaunchKernelGGL((scatter_kernel<T, V, decltype(k)::value, decltype(nt)::value>), dim3((unsigned)blocks), dim3(256), 0, st, a,
                             row_of_slot, static_cast<const T*>(x), weights, static_cast<T*>(rows), row_weights);
        });
      });
    });
  }
  return launched();
}

static int combine_call(int64_t tokens, int32_t topk, int64_t hidden, int32_t dtype, const int32_t* row_of_slot,
                        int64_t num_rows, const void* rows, const float* weights, void* y, int64_t ldy,
                        const float* drow_weights, float* dweights, void* stream) {
  MoveArgs a;
  int rc = check_move(tokens, topk, hidden, dtype, ldy, num_rows, &a);
  if (rc) return rc;
  if ((!row_of_slot || (!rows && num_rows > 0) || !y) && tokens > 0) return fail(MGS_ERR_INVALID_ARG, "row_of_slot, the rows or the token output is NULL");
  if (tokens > 0 && num_rows > 0 && (drow_weights == nullptr) != (dweights == nullptr))
    return fail(MGS_ERR_INVALID_ARG, "drow_weights and dweights go together");
  if (tokens == 0) return ok();
  const bool wide = wide_rows(dtype, hidden, ldy, {rows, y});
  int64_t blocks;
  if ((rc = set_grid(&a, dtype, wide, &blocks))) return rc;
  const int64_t slots = tokens * topk;
  if ((rc = check_overlap({span_rows("the token output", y, tokens, hidden, ldy, dtype), span("dweights", dweights, slots * 4)},
                          {span("row_of_slot", row_of_slot, slots * 4), span_rows("the rows", rows, num_rows, hidden, hidden, dtype),
                           span("weights", weights, slots * 4), span("drow_weights", drow_weights, num_rows * 4)})))
    return rc;
  const hipStream_t st = static_cast<hipStream_t>(stream);
  with_unit(dtype, wide, [&](auto e, auto n) {
    typedef decltype(e) T;
    constexpr int V = decltype(n)::value;
    with_flag(V > 1 && streams(tokens, topk, hidden, dtype), [&](auto nt) {
      with_topk(topk, [&](auto k) {
        hipLaunchKernelGGL((combine_kernel<T, V, decltype(k)::value, decltype(nt)::value>), dim3((unsigned)blocks),
                           dim3(256), 0, st, a, row_of_slot, static_cast<const T*>(rows), weights, static_cast<T*>(y), drow_weights,
                           dweights);
      });
    });
  });
  return launched();
}

int mgs_moe_combine(int64_t tokens, int32_t topk, int64_t hidden, int32_t dtype, const int32_t* row_of_slot,
                    int64_t num_rows, const void* rows, const float* weights, void* y, int64_t ldy, void* stream) {
  return combine_call(tokens, topk, hidden, dtype, row_of_slot, num_rows, rows, weights, y, ldy, nullptr, nullptr, stream);
}

int mgs_moe_dispatch_bwd(int64_t tokens, int32_t topk, int64_t hidden, int32_t dtype, const int32_t* row_of_slot,
                         int64_t num_rows, const void* drows, const float* drow_weights, void* dx, int64_t lddx,
                         float* dweights, void* stream) {
  return combine_call(tokens, topk, hidden, dtype, row_of_slot, num_rows, drows, nullptr, dx, lddx, drow_weights, dweights, stream);
}

int mgs_moe_combine_bwd(int64_t tokens, int32_t topk, int64_t hidden, int32_t dtype, const int32_t* row_of_slot,
                        int64_t num_rows, const void* dy, int64_t lddy, const void* rows, const float* weights,
                        void* drows, float* dweights, void* stream) {
  MoveArgs a;
  int rc = check_move(tokens, topk, hidden, dtype, lddy, num_rows, &a);
  if (rc) return rc;
  if ((!row_of_slot || !dy) && tokens > 0) return fail(MGS_ERR_INVALID_ARG, "row_of_slot or dy is NULL");
  if (!drows && !dweights) {
    if (tokens == 0 || num_rows == 0) return ok();  // (nothing to write, whatever was asked for)
    return fail(MGS_ERR_INVALID_ARG, "no output requested (drows and dweights are NULL)");
  }
  if (dweights && !rows && tokens > 0 && num_rows > 0) return fail(MGS_ERR_INVALID_ARG, "dweights needs rows, the forward's input");
  if (tokens == 0) return ok();
  const bool wide = wide_rows(dtype, hidden, lddy, {dy, rows, drows});
  int64_t blocks;
  if ((rc = set_grid(&a, dtype, wide, &blocks))) return rc;
  const int64_t slots = tokens * topk;
  if ((rc = check_overlap({span_rows("drows", drows, num_rows, hidden, hidden, dtype), span("dweights", dweights, slots * 4)},
                          {span("row_of_slot", row_of_slot, slots * 4), span_rows("dy", dy, tokens, hidden, lddy, dtype),
                           span_rows("rows", rows, num_rows, hidden, hidden, dtype), span("weights", weights, slots * 4)})))
    return rc;
  const hipStream_t st = static_cast<hipStream_t>(stream);
  with_unit(dtype, wide, [&](auto e, auto n) {
    typedef decltype(e) T;
    constexpr int V = decltype(n)::value;
    const dim3 grid((unsigned)blocks);
    with_flag(V > 1 && streams(tokens, topk, hidden, dtype), [&](auto nt) {
      constexpr bool NT = decltype(nt)::value;
      if (!weights && !dweights) {  // without weights the gradient of the rows is a copy
        with_topk(topk, [&](auto k) {
          hipLaunchKernelGGL((scatter_kernel<T, V, decltype(k)::value, NT>), grid, dim3(256), 0, st, a, row_of_slot,
                             static_cast<const T*>(dy), nullptr, static_cast<T*>(drows), nullptr);
        });
      } else {
        hipLaunchKernelGGL((combine_bwd_kernel<T, V, NT>), grid, dim3(256), 0, st, a, row_of_slot, static_cast<const T*>(dy),
                           static_cast<const T*>(rows), weights, static_cast<T*>(drows), dweights);
      }
    });
  });
  return launched();
}

}  // extern "C"
