// Grouped GEMM on MXFP4 operands (E2M1 codes, one E8M0 scale per 32): C_g = A_g . B_g^T with FP32
// accumulation.  Included by gemm_mx.hip, whose tile bookkeeping and epilogue helpers it uses.
//
// The operands go straight into the gfx950 block-scaled MFMA, which takes E2M1 codes and E8M0 scales
// as they are stored.  Operand layout of the 4-bit forms (checked on the device with random codes and
// scales): lane l of the 16 x 16 x 128 form holds row l % 16 and the 32 consecutive K elements of
// block l / 16 in its first four registers, the element with the lower index in the low nibble; its
// scale operand holds that block's scale.  The 32 x 32 x 64 form: row l % 32, K block l / 32.  Products
// of E2M1 values are exact and so were sums over 8192 elements within two binades of scales; over 34
// binades the result was within 1.2e-7 of the 64-bit one (relative 2-norm).

// ---------------------------------------------------------------------------------- few rows
//
// A workgroup owns 16 MT rows x 16 NT columns of one group; its four waves split K: wave w takes the
// 256-element units w, w + 4, ... (a unit of a row is one 128-byte line), and the four partial tiles
// are added in wave order through LDS, so the result does not depend on timing.  Operands go from
// global memory to registers, no LDS staging: with few rows every weight is used by one workgroup only.
template <int MT, int NT>
__global__ __launch_bounds__(256) void gemm_mxfp4_rows_kernel(GemmArgs ga, GemmTable tt) {
  constexpr int TM = 16 * MT, TN = 16 * NT, WAVES = 4;
  __shared__ float part[WAVES][TM][TN + 4];
  int tile;
  TileJob j;
  if (tt.dev) {
    if (!schedule_tile(*tt.dev, blockIdx.x, &tile)) return;
    j = make_job<TM, TN>(ga, *tt.dev, tile);
  } else {
    if (!schedule_tile(tt, blockIdx.x, &tile)) return;
    j = make_job<TM, TN>(ga, tt, tile);
  }
  if (j.k == 0) {
    write_zero_tile<TM, TN>(j, ga);
    return;
  }
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int q = lane >> 4, r16 = lane & 15;
  const fp4_view_t av = fp4_view(j.a.data, j.a.avail), bv = fp4_view(j.b.data, j.b.avail);
  const fp4_view_t asv = fp4_view(j.a.sbase, j.a.savail), bsv = fp4_view(j.b.sbase, j.b.savail);
  v4f acc[MT][NT];
#pragma unroll
  for (int m = 0; m < MT; ++m)
#pragma unroll
    for (int n = 0; n < NT; ++n) acc[m][n] = v4f{0.0f, 0.0f, 0.0f, 0.0f};
  const int nblk = (int)(j.k >> 5);  // 32-element K blocks (k % 32 == 0)
  // the lane's data of fragment row r and K block kb, and its scale; rows past the tile's end and
  // blocks past the end of K read as zero codes with a zero (finite) scale
  auto load = [&](const fp4_view_t& d, const fp4_view_t& s, const Operand& o, int r, int kb, v8i& v, int& sc) {
    const bool ok = r < o.rows && kb < nblk;
    const v4u w = __builtin_amdgcn_raw_buffer_load_b128(d, ok ? r * (int)o.ld + kb * 16 : (int)0x80000000u, 0, 0);
    v = v8i{(int)w[0], (int)w[1], (int)w[2], (int)w[3], 0, 0, 0, 0};
    const uint32_t so = ((uint32_t)(kb >> 2) * (uint32_t)o.srows + (uint32_t)o.srow0 + (uint32_t)r) * 4u + (uint32_t)(kb & 3);
    sc = __builtin_amdgcn_raw_buffer_load_b8(s, ok ? (int)so : (int)0x80000000u, 0, 0);
  };
  for (int u = wave; 8 * u < nblk; u += WAVES) {
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int kb = 8 * u + 4 * h + q;
      v8i a[MT], b[NT];
      int sa[MT], sb[NT];
#pragma unroll
      for (int n = 0; n < NT; ++n) load(bv, bsv, j.b, 16 * n + r16, kb, b[n], sb[n]);
#pragma unroll
      for (int m = 0; m < MT; ++m) load(av, asv, j.a, 16 * m + r16, kb, a[m], sa[m]);
#pragma unroll
      for (int m = 0; m < MT; ++m)
#pragma unroll
        for (int n = 0; n < NT; ++n)
          acc[m][n] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(b[n], a[m], acc[m][n], 4, 4, 0, sb[n], 0, sa[m]);
    }
  }
#pragma unroll
  for (int m = 0; m < MT; ++m)
#pragma unroll
    for (int n = 0; n < NT; ++n)
      *reinterpret_cast<v4f*>(&part[wave][16 * m + r16][16 * n + 4 * q]) = acc[m][n];
  __syncthreads();
  for (int i = threadIdx.x; i < TM * TN / 4; i += 256) {
    const int row = i / (TN / 4), col = 4 * (i - row * (TN / 4));
    if (row >= j.a.rows || col >= j.b.rows) continue;
    v4f s = *reinterpret_cast<const v4f*>(&part[0][row][col]);
#pragma unroll
    for (int w = 1; w < WAVES; ++w) s += *reinterpret_cast<const v4f*>(&part[w][row][col]);
    const uint2 bw = j.bias ? *reinterpret_cast<const uint2*>(j.bias + j.ccol0 + col) : make_uint2(0, 0);
    float v[4];
    frag_values(j, s, bw, v);
    if (j.c32 && ga.accumulate) {
      const float4 o = *reinterpret_cast<const float4*>(j.c32 + (j.crow0 + row) * j.ldc + j.ccol0 + col);
      v[0] += o.x; v[1] += o.y; v[2] += o.z; v[3] += o.w;
    }
    store_values(j, row, col, v);
  }
}
