// Products of BF16 rows with weights held as 4-bit integers in groups, for few rows (decoding), gfx950:
//   w = (q - z) s,   q in 0 .. 15, s BF16 and z in 0 .. 15 (8 without zero points) per group of 32, 64 or 128
//   y[m][n] = sum over groups of s[n][g] (sum_k x[m][k] q[n][k] - z[n][g] sum_k x[m][k])
//
// The time is that of reading the weights once.  They are laid out once in blocks of 16 rows x 128 elements, in the
// order in which a wave's lanes multiply them: a block's codes are 1024 contiguous bytes, 16 a lane, and its scales
// (and zero points) follow.  Lane l = 16 q + r holds row r; its dword j the elements 32 j + 8 q .. + 7, the operand
// of one V_MFMA_F32_16X16X32_BF16, element 2 i in nibble i and element 2 i + 1 in nibble 4 + i, so that a shift, an
// AND and an OR make two BF16 numbers of two codes: the code's bits in the upper mantissa of 16.0 are 16 + q,
// exactly.  The products are summed as they are, and (16 + z) times the sum of the group's x (one more MFMA,
// with ones) is taken off per group before its scale is applied: no weight is ever rounded.  The difference
// loses what the sums' FP32 rounding is of 31 instead of 15 times x: at most 2 (g + 2) 2^-24 31 s sum |x| for a group of
// g elements and scale s, 2^-11 of s sum |x| for g = 128.
// A block of 16 experts x 2 rows, 4096 x 4096, groups of 128, takes 83 us for its 422 MB (5.08 TB/s, a copy's rate); one row of one
// expert and one linear 5.0 us, where a launch and the few loads that a CU has are the time.
// D[row][col] of the MFMA has the first operand's rows: x first, so a lane's four results are four rows m at its own
// weight row, whose scale it holds.
#include <algorithm>
#include <cmath>

#include "launch_size.h"
#include "lds_dma.h"
#include "mgs_device.h"
#include "mgs_span.h"

namespace mgs {
namespace {

typedef unsigned int v4u __attribute__((ext_vector_type(4)));
typedef unsigned int v2u __attribute__((ext_vector_type(2)));
typedef float v4f __attribute__((ext_vector_type(4)));
typedef __bf16 v8bf __attribute__((ext_vector_type(8)));

constexpr int W4_ROWS = 16, W4_K = 128;

// Bytes of a block: codes, then [16 rows][groups] of scales (BF16), or of dwords with the scale in the upper half and
// the BF16 number 16 + z in the lower one.
__host__ __device__ constexpr int w4_block_bytes(int group, bool zeros) {
  return W4_ROWS * W4_K / 2 + W4_ROWS * (W4_K / group) * (zeros ? 4 : 2);
}

struct W4Args {
  const uint16_t* x;
  const uint8_t* w;
  int64_t n, k;       // output columns (the gated form's f), reduction
  int ktiles;         // blocks along k
  int64_t wtiles;     // blocks of rows per expert
  const uint16_t* bias;
  ActArgs act;
  const float* probs;
  void* c;
  int c_f32;
};

template <int G, bool Z>
struct Meta {  // the lane's scales of a block
  v4u d;
  __device__ __forceinline__ void read(const lds8* p) {
    constexpr int B = G * (Z ? 4 : 2);
    if constexpr (B == 2) d[0] = *reinterpret_cast<const __attribute__((address_space(3))) uint16_t*>(p);
    else if constexpr (B == 4) d[0] = *reinterpret_cast<const __attribute__((address_space(3))) uint32_t*>(p);
    else if constexpr (B == 8) {
      const v2u v = *reinterpret_cast<const __attribute__((address_space(3))) v2u*>(p);
      d[0] = v[0]; d[1] = v[1];
    } else {
      d = *reinterpret_cast<const __attribute__((address_space(3))) v4u*>(p);
    }
  }
  __device__ __forceinline__ float scale(int g) const {
    if constexpr (Z) return bf16hi(d[g]);
    else return g & 1 ? bf16hi(d[g >> 1]) : bf16lo(d[g >> 1]);
  }
  __device__ __forceinline__ float zero(int g) const {
    if constexpr (Z) return bf16lo(d[g]);
    else return 24.0f;
  }
};

// two BF16 numbers 16 + q from nibbles i and 4 + i
__device__ __forceinline__ v8bf weights8(uint32_t w) {
  const uint32_t mask = 0x00780078u, one = 0x41804180u;
  v4u r;
  r[0] = ((w << 3) & mask) | one;
  r[1] = ((w >> 1) & mask) | one;
  r[2] = ((w >> 5) & mask) | one;
  r[3] = ((w >> 9) & mask) | one;
  return __builtin_bit_cast(v8bf, r);
}

// A workgroup owns 16 NT weight rows (the gated form: 8 NT gate rows and the same up rows) of one expert and XR of its x
// rows at a time, every `passes`-th such piece (`passes` workgroups share the rows); its waves take the blocks along k
// in turn, each through an LDS ring of D blocks of its own that direct-to-LDS loads fill (weights, scales, and the 128
// elements of each x row that go with them), and wait for the oldest block only.  The partial results are added in wave order through LDS.  Blocks past the end are
// loaded masked, which keeps the wait the same.  G: groups of a block.
template <bool GATED, int XR, int NT, int G, bool Z, int WAVES, int D>
__global__ __launch_bounds__(64 * WAVES) void w4_kernel(W4Args a, GroupTable gt, int passes) {
  constexpr int MT = XR > 16 ? XR / 16 : 1;
  constexpr int BLOCK = w4_block_bytes(W4_K / G, Z), MB = G * (Z ? 4 : 2), TN = GATED ? 8 * NT : 16 * NT;
  constexpr int XAT = NT * 1280, UNIT = XAT + XR * 256, LOADS = 2 * NT + XR / 4;
  constexpr int RING = WAVES * D * UNIT, PART = WAVES * 16 * NT * (16 * MT + 4) * 4;
  __shared__ __attribute__((aligned(1024))) uint8_t smem[RING > PART ? RING : PART];
  auto part = reinterpret_cast<float(*)[16 * NT][16 * MT + 4]>(smem);
  const int ntn = (int)((a.n + TN - 1) / TN);
  const int tiles = ntn * gt.num_groups, pass = blockIdx.x / tiles, tile = blockIdx.x - pass * tiles;
  const int g = tile / ntn, tn = tile - g * ntn;
  const GroupTable& t = gt.dev ? *gt.dev : gt;
  // (wave-uniform, which the compiler cannot tell of a device table's entries: the descriptors are made of them)
  const int64_t r0 = __builtin_amdgcn_readfirstlane(t.row_off[g]), r1 = __builtin_amdgcn_readfirstlane(t.row_off[g + 1]);
  if (r0 + (int64_t)pass * XR >= r1) return;
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int q = lane >> 4, r16 = lane & 15;
  lds8* ring = (lds8*)smem + wave * D * UNIT;
  const uint32_t ring_at = (uint32_t)(uintptr_t)ring;
  // the weight blocks of the workgroup: rows of blocks tn NT .. (gated: tn and its up rows')
  sdesc_t wd[NT];
#pragma unroll
  for (int n = 0; n < NT; ++n) {
    const int64_t half = GATED ? a.n / 16 : a.wtiles;  // blocks of rows of one half
    const int64_t i = GATED ? (int64_t)tn * (NT / 2) + n % (NT / 2) : (int64_t)tn * NT + n;
    const bool there = i < half;
    const int64_t row = GATED && n >= NT / 2 ? half + i : i;
    wd[n] = view(a.w + (g * a.wtiles + (there ? row : 0)) * (int64_t)a.ktiles * BLOCK, there ? (int64_t)a.ktiles * BLOCK : 0);
    desc_final(wd[n]);
  }
  const int64_t ld = 2 * a.k;
  const uint32_t xc = (uint32_t)(((lane & 15) ^ (q << 2)) << 4);  // the chunk that belongs at the lane's position of row 4 i + q
  const bool has_meta = 4 * lane < 16 * MB;
  for (int64_t m0 = r0 + (int64_t)pass * XR; m0 < r1; m0 += (int64_t)passes * XR) {
    const int rows = (int)min<int64_t>(XR, r1 - m0);
    const sdesc_t xd = view(reinterpret_cast<const uint8_t*>(a.x) + m0 * ld, rows * ld);
    desc_final(xd);
    auto issue = [&](int i) {  // the wave's i-th block into slot i % D
      const int kt = wave + WAVES * i;
      const uint32_t dst = ring_at + (uint32_t)(i % D) * UNIT, at = (uint32_t)kt * BLOCK, xk = (uint32_t)kt * 256 + xc;
      const bool in = kt < a.ktiles, xin = in && xk < ld;
#pragma unroll
      for (int n = 0; n < NT; ++n) {
        dma16(wd[n], in ? at + 16u * lane : OUT, dst + n * 1280);
        dma4(wd[n], in && has_meta ? at + 1024u + 4u * lane : OUT, dst + n * 1280 + 1024);
      }
#pragma unroll
      for (int n = 0; n < XR / 4; ++n) dma16(xd, xin ? (uint32_t)((4 * n + q) * ld) + xk : OUT, dst + XAT + n * 1024);
    };
    v4f acc[MT][NT];
#pragma unroll
    for (int m = 0; m < MT; ++m)
#pragma unroll
      for (int n = 0; n < NT; ++n) acc[m][n] = v4f{0.0f, 0.0f, 0.0f, 0.0f};
    const v8bf ones = __builtin_bit_cast(v8bf, v4u{0x3f803f80u, 0x3f803f80u, 0x3f803f80u, 0x3f803f80u});
    const int nb = __builtin_amdgcn_readfirstlane((a.ktiles - wave + WAVES - 1) / WAVES);  // the wave's blocks
#pragma unroll
    for (int i = 0; i < D; ++i) issue(i);
    for (int i = 0; i < nb; ++i) {
      wait_loads<(D - 1) * LOADS>();
      const lds8* u = ring + (i % D) * UNIT;
      v4u wb[NT];
      Meta<G, Z> meta[NT];
#pragma unroll
      for (int n = 0; n < NT; ++n) {
        wb[n] = *reinterpret_cast<const __attribute__((address_space(3))) v4u*>(u + n * 1280 + 16 * lane);
        meta[n].read(u + n * 1280 + 1024 + MB * r16);
      }
      v4u xb[MT][4];
#pragma unroll
      for (int m = 0; m < MT; ++m)
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const int row = (16 * m + r16) & (XR - 1);  // (rows that are not there are multiplied too, and not stored)
          xb[m][j] = *reinterpret_cast<const __attribute__((address_space(3))) v4u*>(
              u + XAT + row * 256 + (((4 * j + q) ^ ((row & 3) << 2)) << 4));
        }
      // the slot is read: refill it
      asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
      issue(i + D);
#pragma unroll
      for (int h = 0; h < G; ++h) {
        v4f p[MT][NT], xs[MT];
#pragma unroll
        for (int m = 0; m < MT; ++m) {
          xs[m] = v4f{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
          for (int n = 0; n < NT; ++n) p[m][n] = v4f{0.0f, 0.0f, 0.0f, 0.0f};
        }
#pragma unroll
        for (int j = 4 / G * h; j < 4 / G * (h + 1); ++j) {
          v8bf wv[NT];
#pragma unroll
          for (int n = 0; n < NT; ++n) wv[n] = weights8(wb[n][j]);
#pragma unroll
          for (int m = 0; m < MT; ++m) {
            const v8bf xv = __builtin_bit_cast(v8bf, xb[m][j]);
            xs[m] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(xv, ones, xs[m], 0, 0, 0);
#pragma unroll
            for (int n = 0; n < NT; ++n) p[m][n] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(xv, wv[n], p[m][n], 0, 0, 0);
          }
        }
#pragma unroll
        for (int n = 0; n < NT; ++n) {
          const float s = meta[n].scale(h), z = meta[n].zero(h);
#pragma unroll
          for (int m = 0; m < MT; ++m)
#pragma unroll
            for (int e = 0; e < 4; ++e)
              acc[m][n][e] = __builtin_fmaf(s, __builtin_fmaf(-z, xs[m][e], p[m][n][e]), acc[m][n][e]);
        }
      }
    }
    wait_loads<0>();
    __syncthreads();
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int m = 0; m < MT; ++m) *reinterpret_cast<v4f*>(&part[wave][16 * n + r16][16 * m + 4 * q]) = acc[m][n];
    __syncthreads();
    for (int i = threadIdx.x; i < TN * 16 * MT; i += 64 * WAVES) {
      const int row = i / TN, col = i - row * TN;
      const int64_t gr = m0 + row, gc = (int64_t)tn * TN + col;
      if (row >= rows || gc >= a.n) continue;
      auto total = [&](int c) {
        float s = part[0][c][row];
#pragma unroll
        for (int w = 1; w < WAVES; ++w) s += part[w][c][row];
        return s;
      };
      float v = total(col);
      if constexpr (GATED) {
        float u = total(TN + col);
        if (a.bias) {
          v += bf16lo(a.bias[g * 2 * a.n + gc]);
          u += bf16lo(a.bias[g * 2 * a.n + a.n + gc]);
        }
        const float s = a.probs ? a.probs[gr] : 1.0f;
        v = (a.act.kind == MGS_ACT_SWIGLU ? act_gated<MGS_ACT_SWIGLU, true>(v, u, a.act)
             : a.act.kind == MGS_ACT_GLU  ? act_gated<MGS_ACT_GLU, true>(v, u, a.act)
                                          : act_gated<MGS_ACT_CLAMPED_SWIGLU, true>(v, u, a.act)) * s;
      } else if (a.bias) {
        v += bf16lo(a.bias[g * a.n + gc]);
      }
      if (a.c_f32) static_cast<float*>(a.c)[gr * a.n + gc] = v;
      else static_cast<uint16_t*>(a.c)[gr * a.n + gc] = (uint16_t)bf16x2(v, 0.0f);
    }
    __syncthreads();  // the partial results are read before the next rows'
  }
}

// ------------------------------------------------------------------------------------- laying out

// One dword of a packed tensor a thread: codes, or a row's scales.
__global__ __launch_bounds__(256) void w4_pack_kernel(int64_t blocks, int64_t wtiles, int ktiles, int64_t n, int64_t k, int group,
                                                      const uint8_t* __restrict__ codes, const uint16_t* __restrict__ scales,
                                                      const uint8_t* __restrict__ zeros, uint8_t* __restrict__ out) {
  const int bytes = w4_block_bytes(group, zeros != nullptr), dw = bytes / 4, G = W4_K / group;
  const int64_t ng = k / group;
  for (int64_t b = blockIdx.x; b < blocks; b += gridDim.x) {
    const int64_t kt = b % ktiles, rt = b / ktiles, e = rt / wtiles, row0 = (rt - e * wtiles) * W4_ROWS;
    uint32_t* o = reinterpret_cast<uint32_t*>(out + b * bytes);
    for (int i = threadIdx.x; i < dw; i += 256) {
      uint32_t v = 0;
      if (i < 256) {
        const int lane = i >> 2, j = i & 3;
        const int64_t row = row0 + (lane & 15), k0 = kt * W4_K + 32 * j + 8 * (lane >> 4);
        if (row < n && k0 < k) {
          const uint8_t* c = codes + ((e * n + row) * k + k0) / 2;
#pragma unroll
          for (int p = 0; p < 4; ++p) v |= (uint32_t)(c[p] & 15) << (4 * p) | (uint32_t)(c[p] >> 4) << (16 + 4 * p);
        }
      } else {
        auto meta = [&](int x) -> uint32_t {  // entry x of the block's [16][G]
          const int64_t row = row0 + x / G, gi = kt * G + x % G;
          if (row >= n || gi >= ng) return zeros ? 0x4180u : 0u;
          const int64_t at = (e * n + row) * ng + gi;
          return zeros ? (uint32_t)scales[at] << 16 | (0x4180u + ((uint32_t)(zeros[at] & 15) << 3)) : scales[at];
        };
        v = zeros ? meta(i - 256) : meta(2 * (i - 256)) | meta(2 * (i - 256) + 1) << 16;
      }
      o[i] = v;
    }
  }
}

// Quantization of BF16 weights, a thread a group (neighbours read 2 g bytes apart: 16 x 8192 x 4096 in groups of 128 take
// 2.9 ms, in groups of 32 0.50 ms; it runs once, on a checkpoint).  With zero points the grid covers [min(w, 0), max(w, 0)] in 15 steps,
// without them it is symmetric in 7 steps each way.  The scale is rounded to BF16 first; codes round to nearest-even
// in steps of the rounded scale.  A group whose scale is 0 has codes equal to its zero point.
__global__ __launch_bounds__(256) void w4_quantize_kernel(int64_t groups, int group, const uint16_t* __restrict__ w,
                                                          uint8_t* __restrict__ codes, uint16_t* __restrict__ scales,
                                                          uint8_t* __restrict__ zeros) {
  for (int64_t i = blockIdx.x * 256ll + threadIdx.x; i < groups; i += gridDim.x * 256ll) {
    const uint16_t* p = w + i * group;
    float lo = 0.0f, hi = 0.0f;
    for (int j = 0; j < group; j += 8) {
      float v[8];
      unpack8(*reinterpret_cast<const uint4*>(p + j), v);
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        lo = fminf(lo, v[e]);
        hi = fmaxf(hi, v[e]);
      }
    }
    // (each half by itself: their difference may overflow)
    const float step = zeros ? hi / 15.0f - lo / 15.0f : fmaxf(hi, -lo) / 7.0f;
    const uint32_t bits = bf16x2(step, 0.0f) & 0xffffu;
    const float s = bf16lo(bits);
    const float z = !zeros ? 8.0f : s > 0.0f ? fminf(rintf(-lo / s), 15.0f) : 0.0f;
    scales[i] = (uint16_t)bits;
    if (zeros) zeros[i] = (uint8_t)z;
    for (int j = 0; j < group; j += 8) {
      float v[8];
      unpack8(*reinterpret_cast<const uint4*>(p + j), v);
      uint32_t c = 0;
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const float f = s > 0.0f ? fminf(fmaxf(rintf(v[e] / s) + z, 0.0f), 15.0f) : z;
        c |= (uint32_t)f << (4 * e);
      }
      *reinterpret_cast<uint32_t*>(codes + (i * group + j) / 2) = c;
    }
  }
}

// ------------------------------------------------------------------------------------------ launches

typedef void (*W4Kernel)(W4Args, GroupTable, int);

template <bool GATED, int MT, int NT, int WAVES, int D>
W4Kernel w4_of(int group, bool zeros) {
  if (zeros)
    return group == 128 ? w4_kernel<GATED, MT, NT, 1, true, WAVES, D>
           : group == 64 ? w4_kernel<GATED, MT, NT, 2, true, WAVES, D> : w4_kernel<GATED, MT, NT, 4, true, WAVES, D>;
  return group == 128 ? w4_kernel<GATED, MT, NT, 1, false, WAVES, D>
         : group == 64 ? w4_kernel<GATED, MT, NT, 2, false, WAVES, D> : w4_kernel<GATED, MT, NT, 4, false, WAVES, D>;
}

// x rows of a pass: the number that needs the least, counting the passes of all groups at what one costs (n = k = 4096,
// 8 or 16 experts, groups of 128, relative to 4 rows: 53 us for a gated pass over 16 experts, 29 us for a plain one).
// Device-resident split sizes: the host knows the capacity only, and takes the groups to be equal.
int pass_rows(const GroupTable& gt) {
  const int xr[4] = {4, 16, 32, 64};
  const double cost[4] = {1.0, 1.05, 1.55, 2.6};
  int best = 4;
  double least = 0.0;
  for (int i = 0; i < 4; ++i) {
    double c = 0.0;
    for (int g = 0; g < gt.num_groups; ++g) {
      const int64_t m = gt.dev ? (gt.total_rows + gt.num_groups - 1) / gt.num_groups : gt.row_off[g + 1] - gt.row_off[g];
      c += cost[i] * (double)((m + xr[i] - 1) / xr[i]);
    }
    if (i == 0 || c < least) {
      least = c;
      best = xr[i];
    }
  }
  return best;
}

// Tile and ring by the pass's rows and by how many blocks of 16 weight rows (the gated form: pairs of them) there are.
// Where these fill the chip, fewer waves a workgroup and more weight rows that share the x rows; where they do not, more
// waves, which split k further.  (us; 16 experts, n = k = 4096, then one expert.)  4 rows: 29.9 with 32 weight rows
// and two waves, 33.9 with 16 and four, 43 with 16 and eight; one expert 6.0 with four waves, 5.0 with eight; gated
// 53 with four waves, 67 with eight.  16 rows: 30.0 with 64 weight rows and two waves, 48 with 16 and four; one
// expert 6.2 with eight waves, 15.6 with 64 weight rows; four experts x 7160 x 2080 in groups of 32 15.3 with 32 weight
// rows and four waves, 17.7 with eight, 18.4 with 16 weight rows; gated 55 with 64, 64 with 32; one expert 7.7 with eight
// waves, 11.8 with two.  32 rows: 22.7 (8 experts) with 64, 31.7 with 32; one expert 6.9 with 16 weight rows and eight
// waves, 11.6 with 64; gated 42 and 52; one expert 8.8 and 13.1.
int w4_launch(const W4Args& a, bool gated, int group, bool zeros, const GroupTable& gt, hipStream_t st) {
  const int xr = pass_rows(gt);
  const int64_t tiles = (a.n + 15) / 16 * gt.num_groups;
  const bool many = tiles >= (gated ? 1024 : 2048), some = tiles >= 512;
  W4Kernel kern;
  int waves = 4, nt = 2;
  if (gated) {
    if (xr == 4) {
      if (many) kern = w4_of<true, 4, 2, 4, 2>(group, zeros);
      else kern = w4_of<true, 4, 2, 8, 2>(group, zeros), waves = 8;
    } else if (xr == 16) {
      if (many) kern = w4_of<true, 16, 4, 4, 1>(group, zeros), nt = 4;
      else kern = w4_of<true, 16, 2, 8, 1>(group, zeros), waves = 8;
    } else if (xr == 32) {
      if (many) kern = w4_of<true, 32, 4, 4, 1>(group, zeros), nt = 4;
      else kern = w4_of<true, 32, 2, 8, 1>(group, zeros), waves = 8;
    } else {
      kern = w4_of<true, 64, 2, 4, 1>(group, zeros);
    }
  } else if (xr == 4) {
    if (many) kern = w4_of<false, 4, 2, 2, 2>(group, zeros), waves = 2;
    else if (some) kern = w4_of<false, 4, 1, 4, 2>(group, zeros), nt = 1;
    else kern = w4_of<false, 4, 1, 8, 2>(group, zeros), nt = 1, waves = 8;
  } else if (xr == 16) {
    if (many) kern = w4_of<false, 16, 4, 2, 2>(group, zeros), nt = 4, waves = 2;
    else if (some) kern = w4_of<false, 16, 2, 4, 1>(group, zeros);
    else kern = w4_of<false, 16, 1, 8, 1>(group, zeros), nt = 1, waves = 8;
  } else if (xr == 32) {
    if (many) kern = w4_of<false, 32, 4, 4, 1>(group, zeros), nt = 4;
    else if (some) kern = w4_of<false, 32, 2, 4, 1>(group, zeros);
    else kern = w4_of<false, 32, 1, 8, 1>(group, zeros), nt = 1, waves = 8;
  } else {
    kern = w4_of<false, 64, 2, 4, 1>(group, zeros);
  }
  const int64_t tn = gated ? 8 * nt : 16 * nt;
  // workgroups that share the passes of a group (61 rows over four experts: 15.3 us, 17.6 in one workgroup each; 512
  // rows of one expert, 4096 x 4096: 38 and 48 us)
  int64_t passes = 1;
  if (gt.dev) passes = gt.total_rows > xr ? 2 : 1;
  else
    for (int g = 0; g < gt.num_groups; ++g) passes = std::max<int64_t>(passes, (gt.row_off[g + 1] - gt.row_off[g] + xr - 1) / xr);
  // (256 experts x 2^20 weight rows, the most that check_w4 takes, are 2^23 workgroups of 256 threads)
  const int64_t base = (a.n + tn - 1) / tn * gt.num_groups;
  passes = shared_passes(passes, base, 64 * waves);
  hipLaunchKernelGGL(kern, dim3((unsigned)(base * passes)), dim3(64 * waves), 0, st, a, gt, (int)passes);
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess) return fail(MGS_ERR_HIP, "HIP launch error: %s", hipGetErrorString(e));
  return ok();
}

int check_w4(int64_t experts, int64_t n, int64_t k, int32_t group) {
  if (experts < 1 || experts > MGS_MAX_GROUPS)
    return fail(MGS_ERR_INVALID_ARG, "num_experts %lld outside [1, %d]", (long long)experts, MGS_MAX_GROUPS);
  if (group != 32 && group != 64 && group != 128) return fail(MGS_ERR_INVALID_ARG, "group %d is not 32, 64 or 128", group);
  if (n < 1 || n > (int64_t)1 << 20) return fail(MGS_ERR_SHAPE, "n = %lld outside [1, 2^20]", (long long)n);
  if (k < 1 || k % group != 0) return fail(MGS_ERR_SHAPE, "k = %lld must be a positive multiple of the group %d", (long long)k, group);
  if (k > (int64_t)1 << 20) return fail(MGS_ERR_SHAPE, "k = %lld is above 2^20", (long long)k);
  return MGS_OK;
}

int64_t w4_nbytes(int64_t experts, int64_t n, int64_t k, int32_t group, bool zeros) {
  return experts * ((n + W4_ROWS - 1) / W4_ROWS) * ((k + W4_K - 1) / W4_K) * w4_block_bytes(group, zeros);
}

int check_w4_call(const mgs_groups* groups, int64_t n_rows, int64_t k, int32_t group, const void* x, const void* w, const void* c,
                  GroupTable* gt, int64_t* rows) {
  int rc = build_groups(groups, gt, rows);
  if (rc) return rc;
  if ((rc = check_w4(gt->num_groups, n_rows, k, group))) return rc;
  if (*rows > 0 && (!x || !w || !c)) return fail(MGS_ERR_INVALID_ARG, "x, w or the output is NULL");
  return MGS_OK;
}

W4Args w4_args(int64_t n, int64_t n_rows, int64_t k, const void* x, const void* w, const void* bias, void* c, bool f32) {
  W4Args a{};
  a.x = static_cast<const uint16_t*>(x);
  a.w = static_cast<const uint8_t*>(w);
  a.n = n;
  a.k = k;
  a.ktiles = (int)((k + W4_K - 1) / W4_K);
  a.wtiles = (n_rows + W4_ROWS - 1) / W4_ROWS;
  a.bias = static_cast<const uint16_t*>(bias);
  a.c = c;
  a.c_f32 = f32;
  return a;
}

}  // namespace
}  // namespace mgs

using namespace mgs;

extern "C" {

int64_t mgs_w4_nbytes(int32_t experts, int64_t n, int64_t k, int32_t group, int32_t zeros) {
  const int rc = check_w4(experts, n, k, group);
  if (rc) return rc;
  ok();
  return w4_nbytes(experts, n, k, group, zeros != 0);
}

int mgs_w4_pack(int32_t experts, int64_t n, int64_t k, int32_t group, const uint8_t* codes, const void* scales_bf16,
                const uint8_t* zeros, void* out, void* stream) {
  int rc = check_w4(experts, n, k, group);
  if (rc) return rc;
  if (!codes || !scales_bf16 || !out) return fail(MGS_ERR_INVALID_ARG, "codes, scales or out is NULL");
  const int64_t groups = experts * n * (k / group), total = w4_nbytes(experts, n, k, group, zeros != nullptr);
  const Range rc_{"codes", codes, experts * n * k / 2}, rs{"scales", scales_bf16, 2 * groups}, rz{"zeros", zeros, groups},
      ro{"out", out, total};
  if ((rc = check_aligned({rs}, 2)) || (rc = check_aligned({ro}, 16))) return rc;
  if ((rc = check_ranges({ro}, {rc_, rs, rz}))) return rc;
  const int64_t wtiles = (n + W4_ROWS - 1) / W4_ROWS, ktiles = (k + W4_K - 1) / W4_K, blocks = experts * wtiles * ktiles;
  hipLaunchKernelGGL(w4_pack_kernel, dim3((unsigned)std::min<int64_t>(blocks, 1 << 20)), dim3(256), 0, static_cast<hipStream_t>(stream),
                     blocks, wtiles, (int)ktiles, n, k, group, codes, static_cast<const uint16_t*>(scales_bf16), zeros,
                     static_cast<uint8_t*>(out));
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess) return fail(MGS_ERR_HIP, "HIP launch error: %s", hipGetErrorString(e));
  return ok();
}

int mgs_w4_quantize(int32_t experts, int64_t n, int64_t k, int32_t group, const void* w_bf16, uint8_t* codes, void* scales_bf16,
                    uint8_t* zeros, void* stream) {
  int rc = check_w4(experts, n, k, group);
  if (rc) return rc;
  if (!w_bf16 || !codes || !scales_bf16) return fail(MGS_ERR_INVALID_ARG, "w, codes or scales is NULL");
  const int64_t groups = experts * n * (k / group);
  const Range rw{"w", w_bf16, 2 * experts * n * k}, rc_{"codes", codes, experts * n * k / 2}, rs{"scales", scales_bf16, 2 * groups},
      rz{"zeros", zeros, groups};
  if ((rc = check_aligned({rw}, 16)) || (rc = check_aligned({rc_}, 4)) || (rc = check_aligned({rs}, 2))) return rc;
  if ((rc = check_ranges({rc_, rs, rz}, {rw}))) return rc;
  hipLaunchKernelGGL(w4_quantize_kernel, dim3((unsigned)std::min<int64_t>((groups + 255) / 256, 1 << 20)), dim3(256), 0,
                     static_cast<hipStream_t>(stream), groups, group, static_cast<const uint16_t*>(w_bf16), codes,
                     static_cast<uint16_t*>(scales_bf16), zeros);
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess) return fail(MGS_ERR_HIP, "HIP launch error: %s", hipGetErrorString(e));
  return ok();
}

int mgs_grouped_gemm_w4(const mgs_groups* groups, int64_t n, int64_t k, int32_t group, int32_t zeros, const void* x_bf16,
                        const void* w, const void* bias_bf16, void* c, int32_t c_dtype, void* stream) {
  if (c_dtype != MGS_DTYPE_BF16 && c_dtype != MGS_DTYPE_F32) return fail(MGS_ERR_INVALID_ARG, "unknown output dtype %d", c_dtype);
  GroupTable gt;
  int64_t rows = 0;
  int rc = check_w4_call(groups, n, k, group, x_bf16, w, c, &gt, &rows);
  if (rc) return rc;
  const bool f32 = c_dtype == MGS_DTYPE_F32;
  const Range rx{"x", x_bf16, 2 * rows * k}, rw{"w", w, w4_nbytes(gt.num_groups, n, k, group, zeros != 0)},
      rb{"bias", bias_bf16, 2 * gt.num_groups * n}, rc_{"c", c, (f32 ? 4 : 2) * rows * n};
  if ((rc = check_aligned({rx, rw}, 16)) || (rc = check_aligned({rb}, 2)) || (rc = check_aligned({rc_}, f32 ? 4 : 2))) return rc;
  if ((rc = check_ranges({rc_}, {rx, rw, rb}))) return rc;
  if (rows == 0) return ok();
  return w4_launch(w4_args(n, n, k, x_bf16, w, bias_bf16, c, f32), false, group, zeros != 0, gt, static_cast<hipStream_t>(stream));
}

int mgs_grouped_gated_w4(const mgs_act_params* act, const mgs_groups* groups, int64_t f, int64_t k, int32_t group, int32_t zeros,
                         const void* x_bf16, const void* w, const void* bias_bf16, const float* probs, void* h_bf16, void* stream) {
  if (!act) return fail(MGS_ERR_INVALID_ARG, "act is NULL");
  if (act->kind != MGS_ACT_SWIGLU && act->kind != MGS_ACT_CLAMPED_SWIGLU && act->kind != MGS_ACT_GLU)
    return fail(MGS_ERR_INVALID_ARG, "activation kind %d is not a gated one", act->kind);
  if (act->kind == MGS_ACT_CLAMPED_SWIGLU &&
      !(act->limit > 0.0f && std::isfinite(act->limit) && std::isfinite(act->alpha) && std::isfinite(act->beta)))
    return fail(MGS_ERR_INVALID_ARG, "CLAMPED_SWIGLU needs a finite limit > 0 and finite alpha, beta");
  if (f < 16 || f % 16 != 0 || f > (int64_t)1 << 19)
    return fail(MGS_ERR_SHAPE, "f = %lld must be a positive multiple of 16 up to 2^19", (long long)f);
  GroupTable gt;
  int64_t rows = 0;
  int rc = check_w4_call(groups, 2 * f, k, group, x_bf16, w, h_bf16, &gt, &rows);
  if (rc) return rc;
  const Range rx{"x", x_bf16, 2 * rows * k}, rw{"w", w, w4_nbytes(gt.num_groups, 2 * f, k, group, zeros != 0)},
      rb{"bias", bias_bf16, 4 * gt.num_groups * f}, rp{"probs", probs, 4 * rows}, rh{"h", h_bf16, 2 * rows * f};
  if ((rc = check_aligned({rx, rw}, 16)) || (rc = check_aligned({rb, rh}, 2)) || (rc = check_aligned({rp}, 4))) return rc;
  if ((rc = check_ranges({rh}, {rx, rw, rb, rp}))) return rc;
  if (rows == 0) return ok();
  W4Args a = w4_args(f, 2 * f, k, x_bf16, w, bias_bf16, h_bf16, false);
  a.act = ActArgs{act->kind, 1.0f, 1.0f, act->limit, act->alpha, act->beta};
  a.probs = probs;
  return w4_launch(a, true, group, zeros != 0, gt, static_cast<hipStream_t>(stream));
}

}  // extern "C"
