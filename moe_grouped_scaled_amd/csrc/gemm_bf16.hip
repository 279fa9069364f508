// Grouped products of unquantized BF16 operands for gfx950, FP32 accumulation, and the gated feed-forward
// block on top of them:
//   FPROP   C_g = A_g . B_g^T      A [M x k], B [E x n x k]          (both operands k-contiguous)
//   DGRAD   C_g = A_g . B_g        A [M x k], B [E x k x n]          (the weight as the forward stores it)
//   WGRAD   C_g = A_g^T . B_g      A [M x m], B [M x n]              (reduction over the group's rows)
//   gated forward   FPROP over [gate | up] rows of the weight; gate and up columns of one tile meet in one
//                   wave, so that the activation and the row's scale are its epilogue
//   gated backward  DGRAD of the second linear; the activation's derivatives are its epilogue
//
// One kernel for all of them: a workgroup of four waves (2 x 2) owns a tile of 64 F x 64 F outputs, each
// wave F x F fragments of V_MFMA_F32_32X32X16_BF16, K steps of 64 elements through a ring of LDS stages that
// direct-to-LDS loads fill.  A k-contiguous operand's stage is rows of 128 bytes (16-byte chunk c of row r at
// position c ^ ((r >> 1) & 7)); the other kind's is the step's 64 rows as they lie in memory, and its
// fragments are read with the transposing LDS read (DS_READ_B64_TR_B16), so that neither a weight nor an
// activation is ever transposed in memory.  Lane layout of that read (checked on the device): in a group of
// 16 lanes, lane s supplies the address of four consecutive elements of row s / 4 and receives column s of the
// group's 16 columns, rows 0..3.  MFMA lane layout: lane l holds row l % 32 of each operand with K elements
// 8 (l / 32) .. + 7; accumulator register r holds D[8 (r / 4) + 4 (l / 32) + r % 4][l % 32].  B is the first
// operand, so a lane's accumulators are columns of one output row.
#include <algorithm>
#include <cmath>
#include <cstring>
#include <type_traits>

#include "launch_size.h"
#include "lds_dma.h"
#include "mgs_device.h"
#include "mgs_span.h"

namespace mgs {
namespace {

typedef int v4i __attribute__((ext_vector_type(4)));
typedef unsigned int v4u __attribute__((ext_vector_type(4)));
typedef float v16f __attribute__((ext_vector_type(16)));
typedef short v4s __attribute__((ext_vector_type(4)));
typedef short v8s __attribute__((ext_vector_type(8)));
typedef __bf16 v8bf __attribute__((ext_vector_type(8)));
typedef __attribute__((address_space(3))) v4s lds_v4s;
typedef __attribute__((address_space(3))) v4i lds_v4i;
typedef float v4f __attribute__((ext_vector_type(4)));
typedef __attribute__((address_space(3))) v4f lds_f4;

enum { EPI_PLAIN = 0, EPI_GATED_FWD = 1, EPI_GATED_BWD = 2 };
constexpr int KSTEP = 64;           // elements of a K step: 128 bytes of a k-contiguous row
constexpr int TILE_BLOCK_N = 4;     // tile columns of a block of the tile order

struct BfArgs {
  int mode;               // mgs_gemm_mode
  int64_t m, n, k;        // n: output columns of the tiles (the gated forward's f)
  const uint16_t* a;
  const uint16_t* b;
  void* c;                // plain: C; gated forward: h [M x n]; gated backward: dpre [M x 2n]
  int c_f32, accumulate;
  const uint16_t* bias;   // plain: [E x n]; gated forward: [E x 2n]
  ActArgs act;
  float lim_in, lim_out;  // clamped SwiGLU: the largest BF16 value at most the limit, the smallest above it
  const float* probs;
  void* pre_out;          // gated forward: [M x 2n], nullable
  const void* pre;        // gated backward: [M x 2n]
  int pre_f32;            // type of either: FP32, or BF16
  uint16_t* h_out;        // gated backward: [M x n], nullable
  float* dp_part;         // gated backward: [M x dp_ld] partial sums of dprobs, nullable
  int64_t dp_ld;
};

// One tile: operand bases and row strides in bytes, the reduction length, the outputs' position.
struct Job {
  int g;
  const uint8_t *a, *b;
  int64_t ald, bld;
  int64_t a_bytes, b_bytes;  // from the base to the operand's end (k-contiguous operands)
  int64_t k;
  int64_t crow0, ccol0;
  int rows, cols, tn;
};

// ---------------------------------------------------------------------------------------- tile order

// The tile workgroup b takes (the schedules of GemmTable); false: none.
template <typename Table>
__device__ __forceinline__ bool schedule_tile(const Table& tt, int b, int* tile) {
  if (!tt.interleave) {
    const int n = tt.total_tiles, q = n >> 3, r = n & 7, x = b & 7, i = b >> 3;
    if (i >= q + (x < r ? 1 : 0)) return false;
    *tile = x * q + min(x, r) + i;
    return true;
  }
  const int s = b / tt.stride;
  if (s >= tt.num_groups) return false;
  const int g = tt.order[s];
  const int j = b - s * tt.stride;
  const int t = tt.tile_off[g + 1] - tt.tile_off[g];
  const int q = t >> 3, r = t & 7, x = j & 7, i = j >> 3;
  if (i >= q + (x < r ? 1 : 0)) return false;
  *tile = tt.tile_off[g] + x * q + min(x, r) + i;
  return true;
}

// TN: output columns of a tile (half the B rows for the gated forward)
template <int MODE, int TM, int TN, typename Table>
__device__ __forceinline__ Job make_job(const BfArgs& ga, const Table& tt, int tile) {
  int lo = 0, hi = tt.num_groups;  // tile_off[lo] <= tile < tile_off[hi]
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (tt.tile_off[mid] <= tile) lo = mid; else hi = mid;
  }
  Job j;
  const int g = lo, lt = tile - tt.tile_off[g];
  j.g = g;
  // tiles of a group run in blocks of TILE_BLOCK_N tile columns, row-major inside a block, so that the
  // workgroups in flight on one XCD share the slices of A and B that its L2 holds
  const int ntn = (int)((ga.n + TN - 1) / TN);
  const int64_t tok0 = tt.tok_off[g], toks = tt.tok_off[g + 1] - tok0;
  const int64_t mrows = MODE == MGS_GEMM_WGRAD ? ga.m : toks;
  const int ntm = (int)((mrows + TM - 1) / TM);
  const int full = ntn / TILE_BLOCK_N, blk = lt / (ntm * TILE_BLOCK_N);
  const int wl = blk < full ? TILE_BLOCK_N : ntn - full * TILE_BLOCK_N;
  const int r = lt - min(blk, full) * ntm * TILE_BLOCK_N;
  const int tm = r / wl, tn = min(blk, full) * TILE_BLOCK_N + (r - tm * wl);
  const int64_t row0 = (int64_t)tm * TM, col0 = (int64_t)tn * TN;
  const uint8_t* a = reinterpret_cast<const uint8_t*>(ga.a);
  const uint8_t* b = reinterpret_cast<const uint8_t*>(ga.b);
  if constexpr (MODE == MGS_GEMM_WGRAD) {
    j.ald = 2 * ga.m;
    j.bld = 2 * ga.n;
    j.a = a + tok0 * j.ald + 2 * row0;
    j.b = b + tok0 * j.bld + 2 * col0;
    j.a_bytes = j.b_bytes = 0;
    j.k = toks;
    j.crow0 = (int64_t)g * ga.m + row0;
  } else {
    j.ald = 2 * ga.k;
    j.a = a + (tok0 + row0) * j.ald;
    j.a_bytes = (toks - row0) * j.ald;
    j.k = ga.k;
    j.crow0 = tok0 + row0;
    if constexpr (MODE == MGS_GEMM_FPROP) {
      j.bld = 2 * ga.k;
      j.b = b + ((int64_t)g * ga.n + col0) * j.bld;  // (the gated forward takes its own)
      j.b_bytes = (ga.n - col0) * j.bld;
    } else {
      j.bld = 2 * ga.n;
      j.b = b + (int64_t)g * ga.k * j.bld + 2 * col0;
      j.b_bytes = 0;
    }
  }
  j.ccol0 = col0;
  j.tn = tn;
  j.rows = (int)min<int64_t>(TM, mrows - row0);
  j.cols = (int)min<int64_t>(TN, ga.n - col0);
  return j;
}

// ------------------------------------------------------------------------------------ loads and MFMAs

// The 4 x 4 fragments of a large tile fill the AGPRs: written as inline assembly, with the accumulators pinned
// there, since the register allocator otherwise keeps part of them elsewhere and spills.  The compiler does not
// see these as MFMAs, so mfma_gap() stands between VALU writes of accumulators and the first one, and
// mfma_drain() between the last one and anything that reads them.
__device__ __forceinline__ void mfma_pinned(v16f& acc, const v4i& b, const v4i& a) {
  asm volatile("v_mfma_f32_32x32x16_bf16 %0, %1, %2, %0" : "+a"(acc) : "v"(b), "v"(a));
}
// the same with a load of 16 bytes a lane behind it, to LDS address `lds` + `off` (M0 is set ahead of the MFMA, which is
// the wait state it needs before the load)
__device__ __forceinline__ void mfma_with_load(v16f& acc, const v4i& b, const v4i& a, const sdesc_t& d, uint32_t voff, uint32_t lds,
                                               int off) {
  asm volatile("s_add_u32 m0, %5, %6\n\tv_mfma_f32_32x32x16_bf16 %0, %1, %2, %0\n\tbuffer_load_dwordx4 %3, %4, 0 offen lds"
               : "+a"(acc) : "v"(b), "v"(a), "v"(voff), "s"(d), "s"(lds), "n"(off) : "memory", "scc");
}
__device__ __forceinline__ void mfma_gap() { asm volatile("s_nop 7"); }
__device__ __forceinline__ void mfma_drain() {
  asm volatile("s_nop 7\n\ts_nop 7\n\ts_nop 7\n\ts_nop 7\n\ts_nop 7\n\ts_nop 7\n\ts_nop 7\n\ts_nop 7");
}

// f(0) .. f(N - 1) with the index a constant: accumulators indexed by a loop that the compiler leaves rolled would go to
// scratch.
template <int N, int I = 0, typename Fn>
__device__ __forceinline__ void unrolled(Fn&& f) {
  if constexpr (I < N) {
    f(std::integral_constant<int, I>{});
    unrolled<N, I + 1>(f);
  }
}

// 16-byte store whose data registers stay live through two wait states (a store wider than 8 bytes reads
// them after it issues)
template <bool NT>
__device__ __forceinline__ void st16(void* p, v4u v) {
  if constexpr (NT) __builtin_nontemporal_store(v, reinterpret_cast<v4u*>(p));
  else *reinterpret_cast<v4u*>(p) = v;
  asm volatile("s_nop 1" ::"v"(v));
}
template <bool NT>
__device__ __forceinline__ void st_f32x8(float* p, const float (&v)[8]) {
  st16<NT>(p, v4u{__float_as_uint(v[0]), __float_as_uint(v[1]), __float_as_uint(v[2]), __float_as_uint(v[3])});
  st16<NT>(p + 4, v4u{__float_as_uint(v[4]), __float_as_uint(v[5]), __float_as_uint(v[6]), __float_as_uint(v[7])});
}
template <bool NT>
__device__ __forceinline__ void st_bf16x8(uint16_t* p, const float (&v)[8]) {
  st16<NT>(p, v4u{bf16x2(v[0], v[1]), bf16x2(v[2], v[3]), bf16x2(v[4], v[5]), bf16x2(v[6], v[7])});
}
__device__ __forceinline__ float act_gated_of(int kind, float g, float u, const ActArgs& aa) {
  return kind == MGS_ACT_SWIGLU ? act_gated<MGS_ACT_SWIGLU, true>(g, u, aa)
         : kind == MGS_ACT_GLU  ? act_gated<MGS_ACT_GLU, true>(g, u, aa)
                                : act_gated<MGS_ACT_CLAMPED_SWIGLU, true>(g, u, aa);
}

// What the backward reads of a gate or an up value: its BF16 rounding, but on the same side of the clamp.  The
// derivative jumps there: rounded to nearest, the values within half a step of the limit (0.1% of them at a limit of
// 1.5 standard deviations) got the other side's derivative, 4% of the gradient in the 2-norm.
__device__ __forceinline__ float same_side(float v, const BfArgs& ga) {
  const float r = bf16lo(bf16x2(v, 0.0f)), m = fabsf(r);  // (NaN stays as it is)
  if (fabsf(v) > ga.act.limit) return m > ga.act.limit ? r : copysignf(ga.lim_out, v);
  return m > ga.act.limit ? copysignf(ga.lim_in, v) : r;
}
// (the gate has no lower clamp: below the limit in magnitude or not, its rounding is on its side)
__device__ __forceinline__ float same_side_gate(float v, const BfArgs& ga) {
  return v > 0.0f ? same_side(v, ga) : v;
}

// One operand of the kernel: the loads of its part of a stage, and its fragments.  T: its rows (outputs) of
// the tile, F = T / 64 fragments a wave, STEP rows apart; KC: k-contiguous; S stages.  Everything that a step's loads and reads need is
// in registers before the loop (lane offsets, LDS addresses of every stage), so that behind an MFMA stand one or two
// instructions: the wave is alone on its SIMD, and what does not fit behind its MFMAs holds them up.
template <int T, bool KC, int S, int STEP>
struct Operand {
  static constexpr int F = T / 64, PITCH = 2 * T;   // bytes of a stage row (not KC)
  static constexpr int LOADS = 2 * F;               // per wave and step
  static constexpr int READS = KC ? F : 2 * F;      // LDS reads of a substep's fragments
  static constexpr int ADDR = KC ? 4 : F;
  uint64_t at;              // the next step's first byte: KC of row 0, else of its first row
  int left;                 // KC: bytes of a row from the next step on; else rows
  int records, ld, col;     // KC: bytes from `at` to the operand's end; not KC: bytes of a row, byte offset in it
  sdesc_t desc;             // of one step
  uint32_t vo[LOADS], ch;   // lane offsets of a step's loads; KC: byte of the lane's chunk in a row (even loads)
  uint32_t dst[S];          // LDS addresses: of the wave's loads, and of the lane's fragments
  uint32_t rd[S][ADDR];

  // row0: the first of the rows that this wave loads (KC); w0: the first of those it multiplies; lds: the operand's
  // part of stage 0, `stage` bytes apart
  __device__ __forceinline__ void init(const uint8_t* p, int64_t ld_, int64_t bytes, int64_t k, int64_t col_, int row0, int w0,
                                       uint32_t lds, uint32_t stage, int wave, int lane) {
    const uint64_t v = reinterpret_cast<uint64_t>(p);
    at = (uint64_t)(uint32_t)__builtin_amdgcn_readfirstlane((uint32_t)(v >> 32)) << 32 | (uint32_t)__builtin_amdgcn_readfirstlane((uint32_t)v);
    ld = __builtin_amdgcn_readfirstlane((int)ld_);
    col = __builtin_amdgcn_readfirstlane((int)col_);
    left = __builtin_amdgcn_readfirstlane((int)(KC ? 2 * k : k));
    records = __builtin_amdgcn_readfirstlane((int)min<int64_t>(bytes, 0x7fffffff));
    const int r32 = lane & 31, h32 = lane >> 5, s4 = (lane & 15) >> 2;
    if constexpr (KC) {
      const int lrow = lane >> 3;
      ch = (uint32_t)(((lane & 7) ^ (lrow >> 1)) << 4);
#pragma unroll
      for (int n = 0; n < LOADS; ++n) vo[n] = (uint32_t)((row0 + 8 * n + lrow) * ld) + (ch ^ (n & 1 ? 64u : 0u));
    } else {
      constexpr int CPR = PITCH / 16, RPI = 1024 / PITCH;  // chunks of a stage row, rows of a load
      const int lr = lane / CPR, pos = lane % CPR;
#pragma unroll
      for (int n = 0; n < LOADS; ++n) {
        const int row = 16 * wave + RPI * n + lr, sw = T == 64 ? (((row >> 1) & 1) << 2) : ((row & 3) << 2);
        vo[n] = (uint32_t)(row * ld) + (uint32_t)((pos ^ sw) << 4);
      }
    }
#pragma unroll
    for (int n = 0; n < LOADS; ++n) asm volatile("" : "+v"(vo[n]));
#pragma unroll
    for (int s = 0; s < S; ++s) {
      dst[s] = __builtin_amdgcn_readfirstlane(lds + s * stage + wave * LOADS * 1024);
#pragma unroll
      for (int i = 0; i < ADDR; ++i) {
        if constexpr (KC) {
          rd[s][i] = lds + s * stage + (uint32_t)(w0 + r32) * 128 + (((2 * i + h32) ^ ((r32 >> 1) & 7)) << 4);
        } else {
          const int chunk = (w0 + STEP * i) / 8 + 2 * ((lane >> 4) & 1) + ((lane & 3) >> 1);
          const int sw = T == 64 ? (((s4 >> 1) & 1) << 2) : (s4 << 2);
          rd[s][i] = lds + s * stage + (uint32_t)((8 * h32 + s4) * PITCH + ((chunk ^ sw) << 4) + 8 * (lane & 1));
        }
        asm volatile("" : "+v"(rd[s][i]));
      }
    }
  }
  // the loads from here on are the next step's (from step 0 on)
  __device__ __forceinline__ void begin() {
    int n;
    if constexpr (KC) {
      n = max(records, 0);
      if (left < 128) {
        // a partial step, and those behind the last: a lane whose chunk is past the row's end stays out from here on
#pragma unroll
        for (int i = 0; i < LOADS; ++i) vo[i] = (int)(ch ^ (i & 1 ? 64u : 0u)) < left ? vo[i] : OUT;
      }
    } else {
      n = left > 0 ? min(left, KSTEP) * ld - col : 0;
    }
    desc = sdesc_t{__builtin_amdgcn_readfirstlane((int)(uint32_t)at), __builtin_amdgcn_readfirstlane((int)((uint32_t)(at >> 32) & 0xffffu)),
                   __builtin_amdgcn_readfirstlane(n), 0x00020000};
    at += KC ? 128 : (uint64_t)KSTEP * (uint32_t)ld;
    left -= KC ? 128 : KSTEP;
    records -= 128;
    desc_final(desc);
  }
  // load n (0 .. LOADS - 1) of the step to stage s
  __device__ __forceinline__ void load(int s, int n) const { dma16(desc, vo[n], dst[s] + n * 1024); }
  // read i (0 .. READS - 1) of the fragments of substep kk of stage s
  __device__ __forceinline__ void read(int s, int kk, int i, v4i (&fr)[F]) const {
    if constexpr (KC) {
      fr[i] = *reinterpret_cast<const lds_v4i*>((lds8*)(uintptr_t)rd[s][kk] + i * STEP * 128);
    } else {
      const int f = i >> 1, h = i & 1;
      const v4s v = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_v4s*)((lds8*)(uintptr_t)rd[s][f] + (16 * kk + 4 * h) * PITCH));
      typedef int v2i __attribute__((ext_vector_type(2)));
      const v2i w = __builtin_bit_cast(v2i, v);
      fr[f][2 * h] = w[0];
      fr[f][2 * h + 1] = w[1];
    }
  }
};

// ------------------------------------------------------------------------------------------ epilogues
//
// A wave's 32 rows at a time go through its part of LDS and leave it by rows, 16 bytes a lane: stored from the
// accumulators, an instruction would write 32 bytes of each of 32 rows.  Lane (r32, h32) holds, for fragment
// (fm, fn) and register group g, row 32 fm + r32 and the four columns 32 fn + 8 g + 4 h32 .. + 3.
// Row fragment fm of the accumulators as 32 FP32 rows.  The 16-byte chunk c of row r stands at position c ^ (r & 15)
// (of the 8 chunks of a 32-column row, F = 1: r & 7), which spreads both the writes, one chunk of every row, and the
// reads, every second chunk of a row, evenly over the banks.
template <int F>
constexpr int STAGED_ROW = 128 * F;
template <int F>
__device__ __forceinline__ lds8* staged(lds8* buf, int row, int chunk) {
  return buf + row * STAGED_ROW<F> + ((chunk ^ (row & (F == 1 ? 7 : 15))) << 4);
}
template <int F>
__device__ __forceinline__ void stage_f32(const v16f (&acc)[F], lds8* buf, int lane) {
  const int r32 = lane & 31, h32 = lane >> 5;
  asm volatile("" ::: "memory");  // a wave's LDS accesses execute in order; this keeps the compiler's order
#pragma unroll
  for (int fn = 0; fn < F; ++fn)
#pragma unroll
    for (int g = 0; g < 4; ++g)
      *reinterpret_cast<lds_f4*>(staged<F>(buf, r32, 8 * fn + 2 * g + h32)) =
          v4f{acc[fn][4 * g], acc[fn][4 * g + 1], acc[fn][4 * g + 2], acc[fn][4 * g + 3]};
  asm volatile("" ::: "memory");
}
// eight columns from col on (a multiple of 8) of a staged row
template <int F>
__device__ __forceinline__ void staged8(lds8* buf, int row, int col, float (&v)[8]) {
  const v4f x = *reinterpret_cast<const lds_f4*>(staged<F>(buf, row, col / 4)), y = *reinterpret_cast<const lds_f4*>(staged<F>(buf, row, col / 4 + 1));
  v[0] = x[0]; v[1] = x[1]; v[2] = x[2]; v[3] = x[3];
  v[4] = y[0]; v[5] = y[1]; v[6] = y[2]; v[7] = y[3];
}
__device__ __forceinline__ void add_bf16x8(float (&v)[8], const uint4& w) {
  v[0] += bf16lo(w.x); v[1] += bf16hi(w.x); v[2] += bf16lo(w.y); v[3] += bf16hi(w.y);
  v[4] += bf16lo(w.z); v[5] += bf16hi(w.z); v[6] += bf16lo(w.w); v[7] += bf16hi(w.w);
}

// [gate | up] of the wave's staged rows in FP32, with their bias: one 16-byte chunk a lane, so that a store writes whole
// lines (with the eight columns a lane of the rows below, two stores write every second chunk each).
template <int F>
__device__ __forceinline__ void pre_f32_rows(const Job& j, const BfArgs& ga, lds8* buf, int row0, int wn, int lane) {
  constexpr int W = 16 * F, LPR = 2 * W / 4, RPP = 64 / LPR;
  const int lr = lane / LPR, c = lane % LPR, half = c / (W / 4), col = wn * W + 4 * (c % (W / 4));
  if (col >= j.cols) return;
  const int64_t gc = half * ga.n + j.ccol0 + col;
  uint2 b = make_uint2(0, 0);
  if (ga.bias) b = *reinterpret_cast<const uint2*>(ga.bias + (int64_t)j.g * 2 * ga.n + gc);
  const v4f add = {bf16lo(b.x), bf16hi(b.x), bf16lo(b.y), bf16hi(b.y)};
#pragma unroll 2
  for (int i = 0; i < 32 / RPP; ++i) {
    const int row = RPP * i + lr;
    if (row0 + row >= j.rows) continue;
    const v4f v = *reinterpret_cast<const lds_f4*>(staged<F>(buf, row, c)) + add;
    st16<F == 4>(static_cast<float*>(ga.pre_out) + (j.crow0 + row0 + row) * 2 * ga.n + gc, __builtin_bit_cast(v4u, v));
  }
}

// The gated forward: a wave's staged rows are 16 F gate columns and the same up columns.  h, and dpre in the backward, leave
// in BF16, one rounding each: the products that take them next multiply BF16 operands, and in FP32 they would be split into
// several.  They are most of the block's error against 64 bits (0.0023 of the 2-norm; with both in FP32 0.0017).
template <int KIND, int F>
__device__ __forceinline__ void gated_fwd_rows(const Job& j, const BfArgs& ga, lds8* buf, int row0, int wn, int lane) {
  constexpr bool NT = F == 4;
  constexpr int W = 16 * F, LPR = W / 8, RPP = 64 / LPR;
  const int lr = lane / LPR, lc = lane % LPR, col = wn * W + 8 * lc;
  if (col >= j.cols) return;
  const int64_t gc = j.ccol0 + col;
  uint4 bg = make_uint4(0, 0, 0, 0), bu = bg;
  if (ga.bias) {
    const uint16_t* b = ga.bias + (int64_t)j.g * 2 * ga.n + gc;
    bg = *reinterpret_cast<const uint4*>(b);
    bu = *reinterpret_cast<const uint4*>(b + ga.n);
  }
#pragma unroll RPP < 32 ? 2 : 1
  for (int i = 0; i < 32 / RPP; ++i) {
    const int row = RPP * i + lr;
    if (row0 + row >= j.rows) continue;
    const int64_t gr = j.crow0 + row0 + row;
    float v[8], u[8], h[8];
    staged8<F>(buf, row, 8 * lc, v);
    staged8<F>(buf, row, W + 8 * lc, u);
    const float s = ga.probs ? ga.probs[gr] : 1.0f;
    add_bf16x8(v, bg);
    add_bf16x8(u, bu);
#pragma unroll
    for (int t = 0; t < 8; ++t) h[t] = act_gated<KIND, true>(v[t], u[t], ga.act) * s;
    st_bf16x8<NT>(static_cast<uint16_t*>(ga.c) + gr * ga.n + gc, h);
    if (ga.pre_out && !ga.pre_f32) {
      if constexpr (KIND == MGS_ACT_CLAMPED_SWIGLU) {
#pragma unroll
        for (int t = 0; t < 8; ++t) {
          v[t] = same_side_gate(v[t], ga);
          u[t] = same_side(u[t], ga);
        }
      }
      uint16_t* p = static_cast<uint16_t*>(ga.pre_out) + gr * 2 * ga.n + gc;
      st_bf16x8<NT>(p, v);
      st_bf16x8<NT>(p + ga.n, u);
    }
  }
}

// The gated backward: da beside what the forward saved of the same eight columns, which is loaded one pass ahead.
template <bool P32>
struct Saved;  // of eight columns: gate, up, and the row's scale
template <>
struct Saved<false> {
  uint4 g, u;
  float s;
  __device__ __forceinline__ void load(const void* p, int64_t at, int64_t n) {
    const uint16_t* q = static_cast<const uint16_t*>(p) + at;
    g = *reinterpret_cast<const uint4*>(q);
    u = *reinterpret_cast<const uint4*>(q + n);
  }
  __device__ __forceinline__ void values(float (&gate)[8], float (&up)[8]) const {
    unpack8(g, gate);
    unpack8(u, up);
  }
};
template <>
struct Saved<true> {
  float4 g0, g1, u0, u1;
  float s;
  __device__ __forceinline__ void load(const void* p, int64_t at, int64_t n) {
    const float* q = static_cast<const float*>(p) + at;
    g0 = *reinterpret_cast<const float4*>(q);
    g1 = *reinterpret_cast<const float4*>(q + 4);
    u0 = *reinterpret_cast<const float4*>(q + n);
    u1 = *reinterpret_cast<const float4*>(q + n + 4);
  }
  __device__ __forceinline__ void values(float (&gate)[8], float (&up)[8]) const {
    gate[0] = g0.x; gate[1] = g0.y; gate[2] = g0.z; gate[3] = g0.w;
    gate[4] = g1.x; gate[5] = g1.y; gate[6] = g1.z; gate[7] = g1.w;
    up[0] = u0.x; up[1] = u0.y; up[2] = u0.z; up[3] = u0.w;
    up[4] = u1.x; up[5] = u1.y; up[6] = u1.z; up[7] = u1.w;
  }
};

template <int KIND, bool P32, int F>
__device__ __forceinline__ void gated_bwd_rows(const Job& j, const BfArgs& ga, lds8* buf, int row0, int wn, int lane) {
  constexpr bool NT = F == 4;
  constexpr int W = 32 * F, LPR = W / 8, RPP = 64 / LPR;
  const int lr = lane / LPR, lc = lane % LPR;
  const bool cok = wn * W + 8 * lc < j.cols;
  const int64_t gc = j.ccol0 + wn * W + 8 * lc, ld = 2 * ga.n, gr0 = j.crow0 + row0;
  auto saved = [&](int row) {
    Saved<P32> x{};
    x.s = 1.0f;
    if (cok && row < 32 && row0 + row < j.rows) {
      x.load(ga.pre, (gr0 + row) * ld + gc, ga.n);
      if (ga.probs) x.s = ga.probs[gr0 + row];
    }
    return x;
  };
  Saved<P32> next = saved(lr);
#pragma unroll 2
  for (int i = 0; i < 32 / RPP; ++i) {
    const int row = RPP * i + lr;
    const Saved<P32> now = next;
    next = saved(row + RPP);
    float v[8], g[8], u[8], dg[8], du[8], h[8], dp = 0.0f;
    staged8<F>(buf, row, 8 * lc, v);
    now.values(g, u);
#pragma unroll
    for (int t = 0; t < 8; ++t) {
      float a, bg, bu;
      dact_gated<KIND, true>(g[t], u[t], ga.act, a, bg, bu);
      dp += v[t] * a;
      const float d = v[t] * now.s;
      dg[t] = d * bg;
      du[t] = d * bu;
      h[t] = a * now.s;
    }
    const bool ok = cok && row0 + row < j.rows;
    const int64_t gr = gr0 + row;
    if (ok) {
      uint16_t* d = static_cast<uint16_t*>(ga.c) + gr * ld + gc;
      st_bf16x8<NT>(d, dg);
      st_bf16x8<NT>(d + ga.n, du);
      if (ga.h_out) st_bf16x8<NT>(ga.h_out + gr * ga.n + gc, h);
    }
    if (ga.dp_part) {
      // over the row's LPR lanes, in a fixed order (columns past the end count nothing)
      dp = ok ? dp : 0.0f;
#pragma unroll
      for (int o = 1; o < LPR; o <<= 1) dp += __shfl_xor(dp, o);
      if (lc == 0 && row0 + row < j.rows) ga.dp_part[gr * ga.dp_ld + 2 * j.tn + wn] = dp;
    }
  }
}

// C with its bias, in BF16 or FP32, optionally added to what is there.
template <bool F32, int F>
__device__ __forceinline__ void plain_rows(const Job& j, const BfArgs& ga, lds8* buf, int row0, int wn, int lane) {
  constexpr bool NT = F == 4;
  constexpr int W = 32 * F, LPR = W / 8, RPP = 64 / LPR;
  const int lr = lane / LPR, lc = lane % LPR, col = wn * W + 8 * lc;
  if (col >= j.cols) return;
  const int64_t gc = j.ccol0 + col;
  uint4 b = make_uint4(0, 0, 0, 0);
  if (ga.bias) b = *reinterpret_cast<const uint4*>(ga.bias + (int64_t)j.g * ga.n + gc);
#pragma unroll 2
  for (int i = 0; i < 32 / RPP; ++i) {
    const int row = RPP * i + lr;
    float v[8];
    staged8<F>(buf, row, 8 * lc, v);
    add_bf16x8(v, b);
    if (row0 + row >= j.rows) continue;
    const int64_t at = (j.crow0 + row0 + row) * ga.n + gc;
    if constexpr (F32) {
      float* c = static_cast<float*>(ga.c) + at;
      if (ga.accumulate) {
        const float4 x = *reinterpret_cast<const float4*>(c), y = *reinterpret_cast<const float4*>(c + 4);
        v[0] += x.x; v[1] += x.y; v[2] += x.z; v[3] += x.w;
        v[4] += y.x; v[5] += y.y; v[6] += y.z; v[7] += y.w;
      }
      st_f32x8<NT>(c, v);
    } else {
      st_bf16x8<NT>(static_cast<uint16_t*>(ga.c) + at, v);
    }
  }
}

template <int EPI, int F, int ACT>
__device__ __forceinline__ void epilogue(const Job& j, const BfArgs& ga, v16f (&acc)[ACT][F], lds8* buf, int wm, int wn, int lane) {
  unrolled<ACT>([&](auto fm_) __attribute__((always_inline)) {
    constexpr int fm = decltype(fm_)::value;
    const int row0 = (2 * fm + wm) * 32;
    if (row0 >= j.rows) return;
    stage_f32<F>(acc[fm], buf, lane);
    if constexpr (EPI == EPI_GATED_FWD) {
      if (ga.pre_out && ga.pre_f32) pre_f32_rows<F>(j, ga, buf, row0, wn, lane);
      if (ga.act.kind == MGS_ACT_SWIGLU) gated_fwd_rows<MGS_ACT_SWIGLU, F>(j, ga, buf, row0, wn, lane);
      else if (ga.act.kind == MGS_ACT_GLU) gated_fwd_rows<MGS_ACT_GLU, F>(j, ga, buf, row0, wn, lane);
      else gated_fwd_rows<MGS_ACT_CLAMPED_SWIGLU, F>(j, ga, buf, row0, wn, lane);
    } else if constexpr (EPI == EPI_GATED_BWD) {
      auto rows = [&](auto p32) __attribute__((always_inline)) {
        constexpr bool P32 = decltype(p32)::value;
        if (ga.act.kind == MGS_ACT_SWIGLU) gated_bwd_rows<MGS_ACT_SWIGLU, P32, F>(j, ga, buf, row0, wn, lane);
        else if (ga.act.kind == MGS_ACT_GLU) gated_bwd_rows<MGS_ACT_GLU, P32, F>(j, ga, buf, row0, wn, lane);
        else gated_bwd_rows<MGS_ACT_CLAMPED_SWIGLU, P32, F>(j, ga, buf, row0, wn, lane);
      };
      if (ga.pre_f32) rows(std::true_type{});
      else rows(std::false_type{});
    } else {
      if (ga.c_f32) plain_rows<true, F>(j, ga, buf, row0, wn, lane);
      else plain_rows<false, F>(j, ga, buf, row0, wn, lane);
    }
  });
}

// ---------------------------------------------------------------------------------------- the kernel

constexpr int stages(int f) { return f == 1 ? 3 : 2; }

// Loop of a K step, in four substeps of 16: a substep's fragments are read from LDS behind the MFMAs of the
// one before, and the step's barrier stands before its last substep, whose fragments are in registers by
// then; behind that substep's MFMAs the next step's first fragments are read, and loads into the stage that
// has just been read begin.  Steps past the end are loaded masked (no memory traffic), which keeps the count of
// loads in flight, and with it each wait, the same for every step.
//
// 256 x 256 tiles need the fewest bytes a product (128 operations a byte from L2) and take a CU's whole register file;
// smaller tiles serve launches that would leave CUs idle (tile_side).  8192 x 8192 x 8192: FPROP, DGRAD and WGRAD 566, 516
// and 523 us on zeros, 760, 756 and 761 us (1.45 PFLOP/s) on random data, which lower the card's clock.  Of FPROP's cycles at
// 8192 x 4096 x 4096 (215 us) 71% are MFMAs, of DGRAD's and WGRAD's 78 to 81%, of the gated forward's (455 us) 66% and of the
// gated backward's (276 us) 55%: the rest are the loads' cycles behind the first and last substep's MFMAs, and each tile's start
// and end (20000 to 33000 cycles), in which all CUs store at a time and none has registers for another tile's products.
template <int MODE, int EPI, int F>
__global__ __launch_bounds__(256) __attribute__((amdgpu_waves_per_eu(F == 4 ? 1 : 2, F == 4 ? 1 : 4)))
void gemm_bf16_kernel(BfArgs ga, GemmTable tt) {
  constexpr int T = 64 * F, S = stages(F), OPB = T * 128, STAGE = 2 * OPB;
  constexpr bool AKC = MODE != MGS_GEMM_WGRAD, BKC = MODE == MGS_GEMM_FPROP;
  constexpr int TN = EPI == EPI_GATED_FWD ? T / 2 : T;
  __shared__ __attribute__((aligned(1024))) uint8_t smem[S * STAGE];
  int tile;
  Job j;
  if (tt.dev) {
    if (!schedule_tile(*tt.dev, blockIdx.x, &tile)) return;
    j = make_job<MODE, T, TN>(ga, *tt.dev, tile);
  } else {
    if (!schedule_tile(tt, blockIdx.x, &tile)) return;
    j = make_job<MODE, T, TN>(ga, tt, tile);
  }
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int wm = wave >> 1, wn = wave & 1;
  lds8* lds = (lds8*)smem;
  const uint32_t lds0 = (uint32_t)(uintptr_t)lds;
  if (MODE == MGS_GEMM_WGRAD && j.k == 0 && ga.accumulate) return;  // an empty group adds nothing

  Operand<T, AKC, S, 64> oa;
  Operand<T, BKC, S, 32> ob;
  oa.init(j.a, j.ald, j.a_bytes, j.k, 2 * (j.crow0 - (MODE == MGS_GEMM_WGRAD ? (int64_t)j.g * ga.m : 0)), 16 * F * wave,
          32 * wm, lds0, STAGE, wave, lane);
  if constexpr (EPI == EPI_GATED_FWD) {
    // B rows of a column wave: 16 F gate rows, then the same 16 F up rows; waves 2w and 2w + 1 load them
    const int half = wave & 1;
    const uint8_t* b = reinterpret_cast<const uint8_t*>(ga.b) + ((int64_t)j.g * 2 * ga.n + half * ga.n + j.ccol0) * j.bld;
    ob.init(b, j.bld, (ga.n - j.ccol0) * j.bld, j.k, 0, 16 * F * (wave >> 1), 32 * F * wn, lds0 + OPB, STAGE, wave, lane);
  } else {
    ob.init(j.b, j.bld, j.b_bytes, j.k, 2 * j.ccol0, 16 * F * wave, 32 * F * wn, lds0 + OPB, STAGE, wave, lane);
  }
  constexpr int NL = 4 * F;
  auto begin = [&]() { oa.begin(); ob.begin(); };
  auto load = [&](int slot, int n) {
    if (n < 2 * F) ob.load(slot, n);
    else oa.load(slot, n - 2 * F);
  };
  v4i fa[2][F], fb[2][F];
  const int nsteps = __builtin_amdgcn_readfirstlane((int)((j.k + KSTEP - 1) / KSTEP));
  // loads into a stage: LEAD of them in the step that frees it, one behind every second MFMA, the others in the
  // next step
  constexpr int LEAD = F == 4 ? 8 : NL;
#pragma unroll
  for (int s = 0; s < S; ++s) {
    begin();
#pragma unroll
    for (int n = 0; n < (s == S - 1 ? LEAD : NL); ++n) load(s, n);
  }
  // The loop over the K steps for the first ACT of the wave's F row fragments.  with(m) says which load (into stage `to`)
  // goes with a substep's m-th MFMA, -1 none; behind(m) comes after it.
  auto run = [&](auto act_) __attribute__((always_inline)) {
    constexpr int ACT = decltype(act_)::value, MFMAS = F * ACT, EVERY = MFMAS / 8;
    constexpr int READS = decltype(ob)::READS + decltype(oa)::READS / F * ACT;
    constexpr int PER = (READS + MFMAS - 1) / MFMAS;  // reads behind each MFMA
    auto read = [&](int slot, int kk, int buf, int i) {
      if (i < decltype(ob)::READS) ob.read(slot, kk, i, fb[buf]);
      else oa.read(slot, kk, i - decltype(ob)::READS, fa[buf]);
    };
    auto reads = [&](int slot, int kk, int buf, int m) {
#pragma unroll
      for (int i = m * PER; i < (m + 1) * PER; ++i)
        if (i < READS) read(slot, kk, buf, i);
    };
    // The accumulators are cleared while the loads are under way, each of its own: of equal values the compiler
    // would keep one and copy it to the others just ahead of their first MFMA, without the wait states.
    v16f acc[ACT][F];
#pragma unroll
    for (int fm = 0; fm < ACT; ++fm)
#pragma unroll
      for (int fn = 0; fn < F; ++fn) {
        acc[fm][fn] = v16f{};
        if constexpr (F == 4) asm volatile("" : "+a"(acc[fm][fn]));
      }
    __builtin_amdgcn_sched_barrier(0);
    mfma_gap();
    __builtin_amdgcn_sched_barrier(0);
    wait_loads<(S - 2) * NL + LEAD>();
    __syncthreads();
    auto substep = [&](int buf, int to, auto&& with, auto&& behind) {
#pragma unroll
      for (int fm = 0; fm < ACT; ++fm)
#pragma unroll
        for (int fn = 0; fn < F; ++fn) {
          const int m = F * fm + fn, n = with(m);
          if constexpr (F == 4) {
            if (n < 0) mfma_pinned(acc[fm][fn], fb[buf][fn], fa[buf][fm]);
            else if (n < 2 * F) mfma_with_load(acc[fm][fn], fb[buf][fn], fa[buf][fm], ob.desc, ob.vo[n & (2 * F - 1)], ob.dst[to], (n & (2 * F - 1)) * 1024);
            else mfma_with_load(acc[fm][fn], fb[buf][fn], fa[buf][fm], oa.desc, oa.vo[n & (2 * F - 1)], oa.dst[to], (n & (2 * F - 1)) * 1024);
          } else {
            acc[fm][fn] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(v8bf, fb[buf][fn]),
                                                                  __builtin_bit_cast(v8bf, fa[buf][fm]), acc[fm][fn], 0, 0, 0);
          }
          behind(m);
          if constexpr (F == 4) __builtin_amdgcn_sched_barrier(0);
        }
    };
    auto none = [](int) { return -1; };
    auto paired = [](int m) { return F == 4 && m % (EVERY ? EVERY : 1) == 0 ? m / (EVERY ? EVERY : 1) : -1; };
    auto step = [&](auto slot_) __attribute__((always_inline)) {
      constexpr int slot = decltype(slot_)::value, prev = slot == 0 ? S - 1 : slot - 1, next = slot == S - 1 ? 0 : slot + 1;
      substep(0, prev, [&](int m) { return LEAD < NL && paired(m) >= 0 ? LEAD + paired(m) : -1; },
              [&](int m) { reads(slot, 1, 1, m); });
      substep(1, 0, none, [&](int m) {
        reads(slot, 2, 0, m);
        if (m == MFMAS - 1) begin();
      });
      substep(0, 0, none, [&](int m) { reads(slot, 3, 1, m); });
      // from here on the next stage is loaded and this one read by every wave
      asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
      wait_loads<(S - 2) * NL>();
      __syncthreads();
      substep(1, slot, paired, [&](int m) {
        reads(next, 0, 0, m);
        if (F != 4 && m == 0) {
#pragma unroll
          for (int n = 0; n < NL; ++n) load(slot, n);
        }
      });
    };
#pragma unroll
    for (int i = 0; i < READS; ++i) read(0, 0, 0, i);
    for (int st = 0; st < nsteps; st += S)
      unrolled<S>([&](auto slot) __attribute__((always_inline)) {
        if (st + decltype(slot)::value < nsteps) step(slot);
      });
    __builtin_amdgcn_sched_barrier(0);
    mfma_drain();
    __builtin_amdgcn_sched_barrier(0);
    __builtin_amdgcn_s_waitcnt(0);  // the masked loads of the steps past the end write LDS too
    __syncthreads();
    lds8* buf = lds + wave * (S * STAGE / 4);
    epilogue<EPI, F, ACT>(j, ga, acc, buf, wm, wn, lane);
  };
  // A group's last tile of at most half the rows leaves out the other row fragments (a wave's fragments are 64 rows apart,
  // so that this halves the work of all four waves): 32 skewed groups, 16384 rows of 7168 x 2048, gated forward without
  // `pre` 1030 -> 1008 us, DGRAD 1000 -> 972; with whole tiles only, nothing changes.
  if (MODE != MGS_GEMM_WGRAD && F > 1 && j.rows <= T / 2) run(std::integral_constant<int, F == 1 ? 1 : F / 2>{});
  else run(std::integral_constant<int, F>{});
}

// ------------------------------------------------------------------------------------------ few rows
//
// With few rows the time is that of reading the weights once, and what counts is bytes in flight.  A
// workgroup owns 16 MT rows x 16 NT weight rows of one group (the gated forward: NT / 2 fragments of gate rows
// and the same of up rows); its WAVES waves split K: wave w takes the 64-element units w, w + WAVES, ..., each wave
// through an LDS ring of D units of its own (a row's unit is one 128-byte line), and waits for the oldest unit
// only.  Waves share nothing until the end, where their partial tiles are added in wave order through LDS, so
// the result does not depend on timing.  Units past the end are loaded masked, which keeps the wait the same.
// Bound by memory: a block of 16 experts x 2 rows, 7168 x 2048, reads its 1.41 GB in 237 us (5.95 TB/s); one row of
// one expert, 4096 x 4096, 14.2 us for 67 MB gated and 9.4 us for 34 MB, of which 3 to 4 us are start and end.
template <int EPI, int XR, int NT, int WAVES, int D>
__global__ __launch_bounds__(64 * WAVES) void rows_bf16_kernel(BfArgs ga, GroupTable gt) {
  constexpr int MT = XR / 16, TB = 16 * NT, TN = EPI == EPI_GATED_FWD ? TB / 2 : TB;
  constexpr int UNIT = NT * 2048 + XR * 128, LOADS = 2 * NT + XR / 8, PITCH = TB + 4;
  constexpr int RING = WAVES * D * UNIT, PART = WAVES * 16 * MT * PITCH * 4;
  __shared__ __attribute__((aligned(1024))) uint8_t smem[RING > PART ? RING : PART];
  const int ntn = (int)((ga.n + TN - 1) / TN);
  const int g = blockIdx.x / ntn, tn = blockIdx.x - g * ntn;
  const GroupTable& t = gt.dev ? *gt.dev : gt;
  const int64_t r0 = __builtin_amdgcn_readfirstlane(t.row_off[g]), r1 = __builtin_amdgcn_readfirstlane(t.row_off[g + 1]);
  if (r0 == r1) return;
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int q = lane >> 4, r16 = lane & 15;
  lds8* lds = (lds8*)smem;
  lds8* ring = lds + wave * D * UNIT;
  const uint32_t ring_at = (uint32_t)(uintptr_t)ring;
  const int64_t ld = 2 * ga.k, col0 = (int64_t)tn * TN;
  const int nunits = __builtin_amdgcn_readfirstlane((int)((ga.k + KSTEP - 1) / KSTEP));
  const int nu = __builtin_amdgcn_readfirstlane((nunits - wave + WAVES - 1) / WAVES);
  // B rows from the tile's first on: one range, or gate and up
  const uint8_t* b = reinterpret_cast<const uint8_t*>(ga.b);
  const int64_t nb = EPI == EPI_GATED_FWD ? 2 * ga.n : ga.n;
  const sdesc_t bd0 = view(b + (g * nb + col0) * ld, (ga.n - col0) * ld);
  const sdesc_t bd1 = EPI == EPI_GATED_FWD ? view(b + (g * nb + ga.n + col0) * ld, (ga.n - col0) * ld) : bd0;
  const int lrow = lane >> 3;
  const uint32_t ch[2] = {(uint32_t)(((lane & 7) ^ (lrow >> 1)) << 4), (uint32_t)(((lane & 7) ^ (lrow >> 1)) << 4) ^ 64u};
  for (int64_t m0 = r0; m0 < r1; m0 += XR) {
    const sdesc_t ad = view(reinterpret_cast<const uint8_t*>(ga.a) + m0 * ld, (r1 - m0) * ld);
    desc_final(ad);
    desc_final(bd0);
    desc_final(bd1);
    auto issue = [&](int i) {  // the wave's i-th unit into slot i % D
      const int64_t k0 = 128 * (int64_t)(wave + WAVES * i);
      const uint32_t dst = ring_at + (uint32_t)(i % D) * UNIT;
      const bool ok[2] = {k0 + ch[0] < ld, k0 + ch[1] < ld};
#pragma unroll
      for (int n = 0; n < 2 * NT; ++n) {
        const int r = EPI == EPI_GATED_FWD ? 8 * (n % NT) + lrow : 8 * n + lrow;
        const uint32_t off = (uint32_t)(r * ld + k0) + ch[n & 1];
        dma16(n < NT ? bd0 : bd1, ok[n & 1] ? off : OUT, dst + n * 1024);
      }
#pragma unroll
      for (int n = 0; n < XR / 8; ++n)
        dma16(ad, ok[n & 1] ? (uint32_t)((8 * n + lrow) * ld + k0) + ch[n & 1] : OUT, dst + (2 * NT + n) * 1024);
    };
    v4f acc[MT][NT];
#pragma unroll
    for (int m = 0; m < MT; ++m)
#pragma unroll
      for (int n = 0; n < NT; ++n) acc[m][n] = v4f{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
    for (int i = 0; i < D; ++i) issue(i);
    for (int i = 0; i < nu; ++i) {
      wait_loads<(D - 1) * LOADS>();
      const lds8* u = ring + (i % D) * UNIT;
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int at = r16 * 128 + (((4 * h + q) ^ ((r16 >> 1) & 7)) << 4);
        v4i bf[NT], af[MT];
#pragma unroll
        for (int n = 0; n < NT; ++n) bf[n] = *reinterpret_cast<const lds_v4i*>(u + n * 2048 + at);
#pragma unroll
        for (int m = 0; m < MT; ++m) af[m] = *reinterpret_cast<const lds_v4i*>(u + NT * 2048 + m * 2048 + at);
#pragma unroll
        for (int m = 0; m < MT; ++m)
#pragma unroll
          for (int n = 0; n < NT; ++n)
            acc[m][n] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(v8bf, bf[n]), __builtin_bit_cast(v8bf, af[m]),
                                                                acc[m][n], 0, 0, 0);
      }
      // the slot's reads are done (the MFMAs have their operands): refill it
      asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
      issue(i + D);
    }
    wait_loads<0>();
    __syncthreads();
    __builtin_amdgcn_sched_barrier(0);
    mfma_drain();
    __builtin_amdgcn_sched_barrier(0);
    auto part = reinterpret_cast<float(*)[16 * MT][PITCH]>(smem);
#pragma unroll
    for (int m = 0; m < MT; ++m)
#pragma unroll
      for (int n = 0; n < NT; ++n)
        *reinterpret_cast<v4f*>(&part[wave][16 * m + r16][16 * n + 4 * q]) = acc[m][n];
    __syncthreads();
    const int rows = (int)min<int64_t>(XR, r1 - m0);
    for (int i = threadIdx.x; i < 16 * MT * TN / 4; i += 64 * WAVES) {
      const int row = i / (TN / 4), col = 4 * (i - row * (TN / 4));
      const int64_t gr = m0 + row, gc = col0 + col;
      if (row >= rows || gc >= ga.n) continue;
      auto total = [&](int c) {
        v4f s = *reinterpret_cast<const v4f*>(&part[0][row][c]);
#pragma unroll
        for (int w = 1; w < WAVES; ++w) s += *reinterpret_cast<const v4f*>(&part[w][row][c]);
        return s;
      };
      auto add_bias = [&](v4f& v, int64_t at) {
        const uint2 bw = *reinterpret_cast<const uint2*>(ga.bias + at);
        v[0] += bf16lo(bw.x); v[1] += bf16hi(bw.x); v[2] += bf16lo(bw.y); v[3] += bf16hi(bw.y);
      };
      auto store = [&](uint16_t* p, v4f v) {
        *reinterpret_cast<uint2*>(p) = make_uint2(bf16x2(v[0], v[1]), bf16x2(v[2], v[3]));
      };
      v4f v = total(col);
      if constexpr (EPI == EPI_PLAIN) {
        if (ga.bias) add_bias(v, g * ga.n + gc);
        if (ga.c_f32) {
          float* c = reinterpret_cast<float*>(ga.c) + gr * ga.n + gc;
          if (ga.accumulate) v += *reinterpret_cast<const v4f*>(c);
          st16<false>(c, __builtin_bit_cast(v4u, v));
        } else {
          store(reinterpret_cast<uint16_t*>(ga.c) + gr * ga.n + gc, v);
        }
      } else {
        v4f u = total(TN + col), h;
        if (ga.bias) {
          add_bias(v, g * nb + gc);
          add_bias(u, g * nb + ga.n + gc);
        }
        const float s = ga.probs ? ga.probs[gr] : 1.0f;
#pragma unroll
        for (int e = 0; e < 4; ++e) h[e] = act_gated_of(ga.act.kind, v[e], u[e], ga.act) * s;
        store(reinterpret_cast<uint16_t*>(ga.c) + gr * ga.n + gc, h);
        if (ga.pre_out && ga.pre_f32) {
          float* p = static_cast<float*>(ga.pre_out) + gr * nb + gc;
          st16<false>(p, __builtin_bit_cast(v4u, v));
          st16<false>(p + ga.n, __builtin_bit_cast(v4u, u));
        } else if (ga.pre_out) {
          if (ga.act.kind == MGS_ACT_CLAMPED_SWIGLU) {
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              v[e] = same_side_gate(v[e], ga);
              u[e] = same_side(u[e], ga);
            }
          }
          uint16_t* p = static_cast<uint16_t*>(ga.pre_out) + gr * nb + gc;
          store(p, v);
          store(p + ga.n, u);
        }
      }
    }
    __syncthreads();  // the partial sums are read before the next rows' loads
  }
}

// dprobs[r] = the sum of the row's partial sums, in order
__global__ __launch_bounds__(256) void dprobs_kernel(GroupTable gt, const float* __restrict__ part, int64_t ld,
                                                     float* __restrict__ dprobs) {
  const int64_t rows = gt.dev ? gt.dev->row_off[gt.num_groups] : gt.total_rows;
  const int64_t r = (int64_t)blockIdx.x * 256 + threadIdx.x;
  if (r >= rows) return;
  float s = 0.0f;
  for (int64_t i = 0; i < ld; ++i) s += part[r * ld + i];
  dprobs[r] = s;
}

// ------------------------------------------------------------------------------------------ tile table

// Tiles of every group and whether a K-grouped launch deals its groups over the XCDs (see GemmTable), from row
// offsets; on the host, or in one thread of gemm_bf16_table_kernel.  A tile's cost is its K steps and about
// eight more for its start and epilogue; where one XCD's contiguous range costs more than 5% above the mean,
// the groups are dealt, the longest first.
__host__ __device__ inline int64_t k_cost(int64_t toks) { return toks ? (toks + KSTEP - 1) / KSTEP + 8 : 1; }

__host__ __device__ inline void fill_table(GemmTable* tt, int e, const int32_t* row_off, bool wgrad, int64_t m, int64_t ntn, int tm) {
  int64_t tiles = 0;
  for (int g = 0; g < e; ++g) {
    tt->tile_off[g] = (int32_t)tiles;
    tt->tok_off[g] = row_off[g];
    tiles += ((wgrad ? m : row_off[g + 1] - row_off[g]) + tm - 1) / tm * ntn;
  }
  tt->tile_off[e] = (int32_t)tiles;
  tt->tok_off[e] = row_off[e];
  tt->num_groups = e;
  tt->total_tiles = (int32_t)tiles;
  tt->interleave = 0;
  tt->stride = 0;
  tt->layout_rows = 0;
  tt->dev = nullptr;
  tt->grid = (int32_t)tiles;
  if (!wgrad || e < 2) return;
  int64_t total = 0, worst = 0;
  for (int g = 0; g < e; ++g) total += k_cost(row_off[g + 1] - row_off[g]) * (tt->tile_off[g + 1] - tt->tile_off[g]);
  const int64_t q = tiles / 8, r = tiles % 8;
  for (int x = 0; x < 8; ++x) {
    const int64_t a = x * q + (x < r ? x : r), b = (x + 1) * q + (x + 1 < r ? x + 1 : r);
    int64_t c = 0;
    for (int g = 0; g < e; ++g) {
      const int64_t lo = a > tt->tile_off[g] ? a : tt->tile_off[g];
      const int64_t hi = b < tt->tile_off[g + 1] ? b : tt->tile_off[g + 1];
      if (hi > lo) c += k_cost(row_off[g + 1] - row_off[g]) * (hi - lo);
    }
    worst = c > worst ? c : worst;
  }
  if (8 * worst * 100 <= total * 105) return;
  tt->interleave = 1;
  tt->stride = (int32_t)((tt->tile_off[1] + 7) / 8 * 8);  // (every group has the same tiles)
  tt->grid = tt->stride * e;
}
// group g's rank by cost, ties in group order
__host__ __device__ inline int k_rank(int g, int e, const int32_t* row_off) {
  const int64_t c = k_cost(row_off[g + 1] - row_off[g]);
  int rank = 0;
  for (int h = 0; h < e; ++h) {
    const int64_t d = k_cost(row_off[h + 1] - row_off[h]);
    rank += (d > c || (d == c && h < g)) ? 1 : 0;
  }
  return rank;
}

__global__ __launch_bounds__(256) void gemm_bf16_table_kernel(const GroupTable* __restrict__ gd, int wgrad, int64_t m,
                                                              int64_t ntn, int tm, GemmTable* __restrict__ out) {
  if (threadIdx.x == 0) fill_table(out, gd->num_groups, gd->row_off, wgrad != 0, m, ntn, tm);
  __syncthreads();
  if (wgrad)
    for (int g = threadIdx.x; g < gd->num_groups; g += 256) out->order[k_rank(g, gd->num_groups, gd->row_off)] = (uint8_t)g;
}

// ------------------------------------------------------------------------------------------ launches

typedef void (*TileKernel)(BfArgs, GemmTable);

template <int MODE, int EPI>
TileKernel tile_kernel(int f) {
  return f == 4 ? gemm_bf16_kernel<MODE, EPI, 4> : f == 2 ? gemm_bf16_kernel<MODE, EPI, 2> : gemm_bf16_kernel<MODE, EPI, 1>;
}

TileKernel tile_kernel_of(int mode, int epi, int f) {
  if (epi == EPI_GATED_FWD) return tile_kernel<MGS_GEMM_FPROP, EPI_GATED_FWD>(f);
  if (epi == EPI_GATED_BWD) return tile_kernel<MGS_GEMM_DGRAD, EPI_GATED_BWD>(f);
  if (mode == MGS_GEMM_FPROP) return tile_kernel<MGS_GEMM_FPROP, EPI_PLAIN>(f);
  if (mode == MGS_GEMM_DGRAD) return tile_kernel<MGS_GEMM_DGRAD, EPI_PLAIN>(f);
  return tile_kernel<MGS_GEMM_WGRAD, EPI_PLAIN>(f);
}

int64_t tile_columns(int epi, int64_t n, int f) {
  const int tn = epi == EPI_GATED_FWD ? 32 * f : 64 * f;
  return (n + tn - 1) / tn;
}

// Tiles of 64 f x 64 f; with device-resident split sizes a bound.
int64_t tile_count(const BfArgs& ga, int epi, const GroupTable& gt, int f) {
  const int tm = 64 * f;
  int64_t rows = 0;
  if (ga.mode == MGS_GEMM_WGRAD) rows = (ga.m + tm - 1) / tm * gt.num_groups;
  else if (gt.dev) rows = ((int64_t)gt.total_rows + tm - 1) / tm + gt.num_groups;
  else
    for (int g = 0; g < gt.num_groups; ++g) rows += (gt.row_off[g + 1] - gt.row_off[g] + tm - 1) / tm;
  return rows * tile_columns(epi, ga.n, f);
}

// The largest group's rows (device-resident split sizes: the host knows the capacity only, and takes the
// largest group to have twice the mean; any other routing is right, if slower)
int64_t most_rows(const GroupTable& gt) {
  if (gt.dev) return std::min<int64_t>(gt.total_rows, std::max<int64_t>(16, 2 * (int64_t)gt.total_rows / gt.num_groups));
  int64_t most = 0;
  for (int g = 0; g < gt.num_groups; ++g) most = std::max<int64_t>(most, gt.row_off[g + 1] - gt.row_off[g]);
  return most;
}

// The largest tiles that the largest group fills by more than half and that give most CUs one: what a larger tile saves
// in loads from L2 and LDS outweighs idle CUs down to about three quarters of the 256 (us, sides 64, 128 and 256).  Plain
// FPROP of 4096 x 4096: 8192 rows (512 tiles of 256) 393, 257, 210; 1024 rows (64 tiles of 256, 256 of 128) 53, 43, 72;
// 512 rows (32 and 128) 28, 40, 72.  WGRAD of 4096 x 4096 over 512 rows (256 and 1024) 38, 27, 22; of 4096 x 2048 over
// 2048 rows (128 and 512) 55, 38, 44.  Small groups lose little to half-empty tiles: 16 skewed groups, 1024 rows of
// 7168 x 2048, FPROP 123, 119, 124, DGRAD 255, 197, 207.
int tile_side(const BfArgs& ga, int epi, const GroupTable& gt) {
  const int64_t side = ga.mode == MGS_GEMM_WGRAD ? ga.m : most_rows(gt);
  if (side > 128 && tile_count(ga, epi, gt, 4) >= 192) return 4;
  if (side > 64 && tile_count(ga, epi, gt, 2) >= 192) return 2;
  return 1;
}

// Whether workgroups of 32 weight rows (the gated form: of 16 pairs) leave CUs without two of them.
bool few_tiles(const BfArgs& ga, int epi, const GroupTable& gt) {
  const int64_t tn = epi == EPI_GATED_FWD ? 16 : 32;
  return (ga.n + tn - 1) / tn * gt.num_groups < 512;
}

// x rows of a workgroup of the kernel for few rows, or 0 where the tiles are faster.  (us, gated and plain.)  One expert,
// 4096 x 4096: 32 rows 13.8 and 10.5, 64 rows 17.0 and 11.0, on tiles 20.8 and 18.2, which 128 rows take too.  16
// experts, 7168 x 2048: 2 rows each 153 and 82, 32 rows 162 and 90, on tiles 168 and 87; 64 rows 188 and 102, on
// tiles 186 and 101.  With few workgroups the weight rows of one are fewer, so that more CUs read (one row, plain:
// 9.4 against 12.2); with many and 32 rows they are more, so that the x rows are read less often (162 against 183).
int few_rows(const BfArgs& ga, int epi, const GroupTable& gt) {
  if (ga.mode != MGS_GEMM_FPROP) return 0;
  const int64_t most = most_rows(gt);
  return most <= 16 ? 16 : most <= 32 ? 32 : most <= 64 && few_tiles(ga, epi, gt) ? 64 : 0;
}

// Enqueues the product (the device table first, where
// the split sizes are device-resident).
int launch(const BfArgs& ga, int epi, const GroupTable& gt, GemmTable* dev_table, hipStream_t st) {
  if (const int xr = few_rows(ga, epi, gt)) {
    const bool gated = epi == EPI_GATED_FWD, few = few_tiles(ga, epi, gt);
    void (*kern)(BfArgs, GroupTable);
    int waves = 4, tn = 32;
    if (gated) {
      tn = 16;
      if (xr == 16) kern = rows_bf16_kernel<EPI_GATED_FWD, 16, 2, 4, 2>;
      else if (xr == 64) kern = rows_bf16_kernel<EPI_GATED_FWD, 64, 2, 4, 1>;
      else if (few) kern = rows_bf16_kernel<EPI_GATED_FWD, 32, 2, 4, 2>;
      else kern = rows_bf16_kernel<EPI_GATED_FWD, 32, 4, 4, 1>, tn = 32;
    } else if (few) {
      tn = 16;
      if (xr == 16) kern = rows_bf16_kernel<EPI_PLAIN, 16, 1, 8, 2>, waves = 8;
      else if (xr == 32) kern = rows_bf16_kernel<EPI_PLAIN, 32, 1, 8, 2>, waves = 8;
      else kern = rows_bf16_kernel<EPI_PLAIN, 64, 1, 4, 2>;
    } else {
      if (xr == 16) kern = rows_bf16_kernel<EPI_PLAIN, 16, 2, 4, 2>;
      else kern = rows_bf16_kernel<EPI_PLAIN, 32, 4, 4, 1>, tn = 64;
    }
    const int64_t grid = (int64_t)gt.num_groups * ((ga.n + tn - 1) / tn);
    // (beyond: only the gated form of 256 experts x 2^20 pairs)
    if (grid > most_workgroups(64 * waves)) return fail(MGS_ERR_SHAPE, "too many tiles");
    hipLaunchKernelGGL(kern, dim3((unsigned)grid), dim3(64 * waves), 0, st, ga, gt);
  } else {
    const int f = tile_side(ga, epi, gt), tm = 64 * f;
    const int64_t ntn = tile_columns(epi, ga.n, f), tiles = tile_count(ga, epi, gt, f);
    const bool wgrad = ga.mode == MGS_GEMM_WGRAD;
    // (dealing the groups of a K-grouped launch rounds each up to a multiple of 8 workgroups)
    if (tiles + 8 * ((int64_t)gt.num_groups + 1) > INT32_MAX / 256) return fail(MGS_ERR_SHAPE, "too many tiles");
    GemmTable tt{};
    if (gt.dev) {
      hipLaunchKernelGGL(gemm_bf16_table_kernel, dim3(1), dim3(256), 0, st, gt.dev, wgrad ? 1 : 0, ga.m, ntn, tm, dev_table);
      tt.dev = dev_table;
      // per-XCD rounding of either schedule
      tt.grid = (int32_t)(wgrad ? (int64_t)gt.num_groups * ((tiles / gt.num_groups + 7) / 8 * 8) + 8 : tiles + 8);
    } else {
      fill_table(&tt, gt.num_groups, gt.row_off, wgrad, ga.m, ntn, tm);
      if (tt.interleave)
        for (int g = 0; g < gt.num_groups; ++g) tt.order[k_rank(g, gt.num_groups, gt.row_off)] = (uint8_t)g;
      if (tt.total_tiles == 0) return ok();
    }
    hipLaunchKernelGGL(tile_kernel_of(ga.mode, epi, f), dim3((unsigned)tt.grid), dim3(256), 0, st, ga, tt);
  }
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess) return fail(MGS_ERR_HIP, "HIP launch error: %s", hipGetErrorString(e));
  return ok();
}

// Widths of rows in memory: whole 16-byte units, and 256 rows within 32-bit offsets.
int check_bf16_width(int64_t w, const char* what) {
  if (w <= 0 || w % 8 != 0) return fail(MGS_ERR_SHAPE, "%s = %lld must be a positive multiple of 8", what, (long long)w);
  if (w > (int64_t)1 << 20) return fail(MGS_ERR_SHAPE, "%s = %lld is above 2^20", what, (long long)w);
  return MGS_OK;
}

int check_gated(const mgs_act_params* act, ActArgs* out) {
  if (!act) return fail(MGS_ERR_INVALID_ARG, "act is NULL");
  if (act->kind != MGS_ACT_SWIGLU && act->kind != MGS_ACT_CLAMPED_SWIGLU && act->kind != MGS_ACT_GLU)
    return fail(MGS_ERR_INVALID_ARG, "activation kind %d is not a gated one", act->kind);
  if (act->kind == MGS_ACT_CLAMPED_SWIGLU &&
      !(act->limit > 0.0f && std::isfinite(act->limit) && std::isfinite(act->alpha) && std::isfinite(act->beta)))
    return fail(MGS_ERR_INVALID_ARG, "CLAMPED_SWIGLU needs a finite limit > 0 and finite alpha, beta");
  *out = ActArgs{act->kind, 1.0f, 1.0f, act->limit, act->alpha, act->beta};
  return MGS_OK;
}

int check_pre_dtype(int32_t dtype) {
  if (dtype != MGS_DTYPE_BF16 && dtype != MGS_DTYPE_F32) return fail(MGS_ERR_INVALID_ARG, "unknown type of pre %d", dtype);
  return MGS_OK;
}

int64_t dp_columns(int64_t f) { return 2 * ((f + 63) / 64); }  // partial sums of a row (64-wide tiles have the most)

}  // namespace
}  // namespace mgs

using namespace mgs;

extern "C" {

int mgs_grouped_gemm_bf16(int32_t mode, const mgs_groups* groups, int64_t m, int64_t n, int64_t k, const void* a_bf16,
                          const void* b_bf16, void* c, int32_t c_dtype, const void* bias_bf16, int32_t accumulate,
                          void* stream) {
  if (mode != MGS_GEMM_FPROP && mode != MGS_GEMM_DGRAD && mode != MGS_GEMM_WGRAD)
    return fail(MGS_ERR_INVALID_ARG, "unknown GEMM mode %d", mode);
  if (c_dtype != MGS_DTYPE_BF16 && c_dtype != MGS_DTYPE_F32) return fail(MGS_ERR_INVALID_ARG, "unknown output dtype %d", c_dtype);
  if (accumulate && c_dtype != MGS_DTYPE_F32) return fail(MGS_ERR_UNSUPPORTED, "accumulate needs an FP32 output");
  GroupTable gt;
  int64_t rows = 0;
  int rc = build_groups(groups, &gt, &rows);
  if (rc) return rc;
  if ((rc = check_bf16_width(n, "n"))) return rc;
  const int64_t e = gt.num_groups;
  const bool wgrad = mode == MGS_GEMM_WGRAD;
  if ((rc = check_bf16_width(wgrad ? m : k, wgrad ? "m" : "k"))) return rc;
  if ((wgrad ? k : m) != rows)
    return fail(MGS_ERR_SHAPE, "%s = %lld must equal the split sum %lld", wgrad ? "k" : "m", (long long)(wgrad ? k : m), (long long)rows);
  if (bias_bf16 && wgrad) return fail(MGS_ERR_INVALID_ARG, "bias is not defined for WGRAD");
  if (!c && (rows > 0 || wgrad)) return fail(MGS_ERR_INVALID_ARG, "c is NULL");
  if (rows > 0 && (!a_bf16 || !b_bf16)) return fail(MGS_ERR_INVALID_ARG, "operand %s is NULL", a_bf16 ? "b" : "a");
  const Range ra{"a", a_bf16, 2 * rows * (wgrad ? m : k)}, rb{"b", b_bf16, 2 * n * (wgrad ? rows : e * k)},
      rc_{"c", c, (c_dtype == MGS_DTYPE_F32 ? 4 : 2) * n * (wgrad ? e * m : rows)}, rbias{"bias", bias_bf16, 2 * e * n};
  if ((rc = check_aligned({ra, rb, rc_, rbias}, 16))) return rc;
  if ((rc = check_ranges({rc_}, {ra, rb, rbias}))) return rc;
  if (rows == 0 && !wgrad) return ok();
  BfArgs ga{};
  ga.mode = mode;
  ga.m = m; ga.n = n; ga.k = k;
  ga.a = static_cast<const uint16_t*>(a_bf16);
  ga.b = static_cast<const uint16_t*>(b_bf16);
  ga.c = c;
  ga.c_f32 = c_dtype == MGS_DTYPE_F32;
  ga.accumulate = accumulate != 0;
  ga.bias = static_cast<const uint16_t*>(bias_bf16);
  return launch(ga, EPI_PLAIN, gt, dev_gemm_table(groups), static_cast<hipStream_t>(stream));
}

int mgs_grouped_gated_fwd(const mgs_act_params* act, const mgs_groups* groups, int64_t f, int64_t k, const void* x_bf16,
                          const void* w_bf16, const void* bias_bf16, const float* probs, void* h_bf16, void* pre,
                          int32_t pre_dtype, void* stream) {
  BfArgs ga{};
  int rc = check_gated(act, &ga.act);
  if (rc) return rc;
  GroupTable gt;
  int64_t rows = 0;
  if ((rc = build_groups(groups, &gt, &rows))) return rc;
  if ((rc = check_bf16_width(f, "f")) || (rc = check_bf16_width(k, "k"))) return rc;
  if (pre && (rc = check_pre_dtype(pre_dtype))) return rc;
  if (rows > 0 && (!x_bf16 || !w_bf16 || !h_bf16)) return fail(MGS_ERR_INVALID_ARG, "x, w or h is NULL");
  const int64_t e = gt.num_groups;
  const Range rx{"x", x_bf16, 2 * rows * k}, rw{"w", w_bf16, 4 * e * f * k}, rbias{"bias", bias_bf16, 4 * e * f},
      rp{"probs", probs, 4 * rows}, rh{"h", h_bf16, 2 * rows * f}, rpre{"pre", pre, (pre_dtype == MGS_DTYPE_F32 ? 8 : 4) * rows * f};
  if ((rc = check_aligned({rx, rw, rbias, rh, rpre}, 16)) || (rc = check_aligned({rp}, 4))) return rc;
  if ((rc = check_ranges({rh, rpre}, {rx, rw, rbias, rp}))) return rc;
  if (rows == 0) return ok();
  if (ga.act.kind == MGS_ACT_CLAMPED_SWIGLU) {
    uint32_t bits;
    std::memcpy(&bits, &ga.act.limit, 4);  // finite and positive: truncation rounds down, one step up is above
    const uint32_t in = bits & 0xffff0000u, out = in + 0x10000u;
    std::memcpy(&ga.lim_in, &in, 4);
    std::memcpy(&ga.lim_out, &out, 4);
  }
  ga.mode = MGS_GEMM_FPROP;
  ga.m = rows; ga.n = f; ga.k = k;
  ga.a = static_cast<const uint16_t*>(x_bf16);
  ga.b = static_cast<const uint16_t*>(w_bf16);
  ga.c = h_bf16;
  ga.bias = static_cast<const uint16_t*>(bias_bf16);
  ga.probs = probs;
  ga.pre_out = pre;
  ga.pre_f32 = pre_dtype == MGS_DTYPE_F32;
  return launch(ga, EPI_GATED_FWD, gt, dev_gemm_table(groups), static_cast<hipStream_t>(stream));
}

int64_t mgs_grouped_gated_bwd_workspace_bytes(const mgs_groups* groups, int64_t f) {
  GroupTable gt;
  int64_t rows = 0;
  int rc = build_groups(groups, &gt, &rows);
  if (rc) return rc;
  if ((rc = check_bf16_width(f, "f"))) return rc;
  ok();
  return 4 * rows * dp_columns(f);
}

int mgs_grouped_gated_bwd(const mgs_act_params* act, const mgs_groups* groups, int64_t f, int64_t n, const void* dy_bf16,
                          const void* w2_bf16, const void* pre, int32_t pre_dtype, const float* probs, void* dpre_bf16,
                          void* h_bf16, float* dprobs, void* workspace, int64_t workspace_bytes, void* stream) {
  BfArgs ga{};
  int rc = check_gated(act, &ga.act);
  if (rc) return rc;
  GroupTable gt;
  int64_t rows = 0;
  if ((rc = build_groups(groups, &gt, &rows))) return rc;
  if ((rc = check_bf16_width(f, "f")) || (rc = check_bf16_width(n, "n"))) return rc;
  if ((rc = check_pre_dtype(pre_dtype))) return rc;
  if (rows > 0 && (!dy_bf16 || !w2_bf16 || !pre || !dpre_bf16)) return fail(MGS_ERR_INVALID_ARG, "dy, w2, pre or dpre is NULL");
  const int64_t e = gt.num_groups, need = dprobs ? 4 * rows * dp_columns(f) : 0;
  if (need > 0 && (!workspace || workspace_bytes < need))
    return fail(MGS_ERR_INVALID_ARG, "dprobs needs a workspace of %lld bytes (got %lld%s)", (long long)need,
                (long long)workspace_bytes, workspace ? "" : ", NULL");
  const Range rdy{"dy", dy_bf16, 2 * rows * n}, rw{"w2", w2_bf16, 2 * e * n * f}, rpre{"pre", pre, (pre_dtype == MGS_DTYPE_F32 ? 8 : 4) * rows * f},
      rp{"probs", probs, 4 * rows}, rd{"dpre", dpre_bf16, 4 * rows * f}, rh{"h", h_bf16, 2 * rows * f},
      rdp{"dprobs", dprobs, 4 * rows}, rws{"the workspace", need ? workspace : nullptr, need};
  if ((rc = check_aligned({rdy, rw, rpre, rd, rh}, 16)) || (rc = check_aligned({rp, rdp, rws}, 4))) return rc;
  if ((rc = check_ranges({rd, rh, rdp, rws}, {rdy, rw, rpre, rp}))) return rc;
  if (rows == 0) return ok();
  ga.mode = MGS_GEMM_DGRAD;
  ga.m = rows; ga.n = f; ga.k = n;
  ga.a = static_cast<const uint16_t*>(dy_bf16);
  ga.b = static_cast<const uint16_t*>(w2_bf16);
  ga.c = dpre_bf16;
  ga.pre = pre;
  ga.pre_f32 = pre_dtype == MGS_DTYPE_F32;
  ga.h_out = static_cast<uint16_t*>(h_bf16);
  ga.probs = probs;
  const hipStream_t st = static_cast<hipStream_t>(stream);
  if (dprobs) {
    const int64_t side = 64 * tile_side(ga, EPI_GATED_BWD, gt);
    ga.dp_part = static_cast<float*>(workspace);
    ga.dp_ld = 2 * ((f + side - 1) / side);
  }
  if ((rc = launch(ga, EPI_GATED_BWD, gt, dev_gemm_table(groups), st))) return rc;
  if (!dprobs) return rc;
  hipLaunchKernelGGL(dprobs_kernel, dim3((unsigned)((rows + 255) / 256)), dim3(256), 0, st, gt, ga.dp_part, ga.dp_ld, dprobs);
  const hipError_t err = hipGetLastError();
  if (err != hipSuccess) return fail(MGS_ERR_HIP, "HIP launch error: %s", hipGetErrorString(err));
  return ok();
}

}  // extern "C"
