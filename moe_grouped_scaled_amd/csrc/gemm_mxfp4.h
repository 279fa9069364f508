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
// 256-element units w, w + 4, ... and the four partial tiles are added in wave order through LDS, so the
// result does not depend on timing.  With few rows the time is that of reading the weights once, so what
// counts is bytes in flight: every wave has its own ring of D units in LDS, filled by direct-to-LDS loads
// (eight lanes read a row's 128-byte line; reading fragments from global memory straight into registers,
// four rows per lane quad, reached 4.0 TB/s), and waits for the oldest unit only.  Waves share nothing
// until the end: no barrier in the loop.  Units past the end are loaded masked (no memory traffic), which
// keeps the count of loads in flight, and with it the wait, the same for every unit.
typedef int v4i __attribute__((ext_vector_type(4)));

constexpr int rows_scale_loads(int frags) { return (32 * frags + 63) / 64; }  // dword loads, 64 lanes each
constexpr int rows_unit_bytes(int mt, int nt) {
  return (mt + nt) * 2048 + (rows_scale_loads(mt) + rows_scale_loads(nt)) * 256;
}

template <int N>
__device__ __forceinline__ void wait_loads() { asm volatile("s_waitcnt vmcnt(%0)" ::"n"(N) : "memory"); }

template <int MT, int NT, int D>
__global__ __launch_bounds__(256) void gemm_mxfp4_rows_kernel(GemmArgs ga, GemmTable tt) {
  constexpr int TM = 16 * MT, TN = 16 * NT, WAVES = 4;
  constexpr int SM = rows_scale_loads(MT), SN = rows_scale_loads(NT), UNIT = rows_unit_bytes(MT, NT);
  constexpr int LOADS = 2 * (MT + NT) + SM + SN;  // per unit
  constexpr int PITCH = TN + 4;
  constexpr int RING = WAVES * D * UNIT, PART = WAVES * TM * PITCH * 4;
  __shared__ __attribute__((aligned(1024))) uint8_t smem[RING > PART ? RING : PART];
  int tile;
  TileJob j;
  if (tt.dev) {
    if (!schedule_tile(*tt.dev, blockIdx.x, &tile)) return;
    j = make_job<MGS_FMT_MXFP4, TM, TN>(ga, *tt.dev, tile);
  } else {
    if (!schedule_tile(tt, blockIdx.x, &tile)) return;
    j = make_job<MGS_FMT_MXFP4, TM, TN>(ga, tt, tile);
  }
  if (j.k == 0) {
    write_zero_tile<TM, TN>(j, ga);
    return;
  }
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int q = lane >> 4, r16 = lane & 15;
  const int nblk = __builtin_amdgcn_readfirstlane((int)(j.k >> 5));  // 32-element K blocks (k % 32 == 0)
  const int nslices = (nblk + 3) >> 2;
  const sdesc_t ad = gemm_view(j.a.data, j.a.avail), bd = gemm_view(j.b.data, j.b.avail);
  const sdesc_t as = gemm_view(j.a.sbase, j.a.savail), bs = gemm_view(j.b.sbase, j.b.savail);
  const uint32_t as4 = __builtin_amdgcn_readfirstlane((uint32_t)j.a.srows * 4u), bs4 = __builtin_amdgcn_readfirstlane((uint32_t)j.b.srows * 4u);
  constexpr uint32_t OUT = 0x80000000u;  // past every record count: reads as zero, no memory access
  // data load: row 8 i + lane / 8 of a fragment set, the chunk that belongs at position lane % 8
  const int lrow = lane >> 3, chunk = (lane & 7) ^ lrow;
  const uint32_t ald = (uint32_t)j.a.ld, bld = (uint32_t)j.b.ld;
  uint8_t* ring = smem + wave * D * UNIT;
  const uint32_t ring_at = lds_addr(ring);
  auto issue = [&](int i) {  // the wave's i-th unit into slot i % D
    const int u = wave + WAVES * i;
    const uint32_t base = ring_at + (uint32_t)(i % D) * UNIT;
    const bool cok = 8 * u + chunk < nblk;
    const uint32_t k0 = 128u * (uint32_t)u + 16u * (uint32_t)chunk;
#pragma unroll
    for (int n = 0; n < 2 * NT; ++n) {
      const int r = 8 * n + lrow;
      dma16(bd, cok && r < j.b.rows ? (uint32_t)r * bld + k0 : OUT, 0, base + n * 1024);
    }
#pragma unroll
    for (int n = 0; n < SN; ++n) {
      const int x = 64 * n + lane, sl = x / TN, r = x - sl * TN;
      const bool ok = sl < 2 && 2 * u + sl < nslices && r < j.b.rows;
      dma4(bs, ok ? (uint32_t)(2 * u + sl) * bs4 + ((uint32_t)j.b.srow0 + (uint32_t)r) * 4u : OUT, 0, base + NT * 2048 + n * 256);
    }
#pragma unroll
    for (int n = 0; n < 2 * MT; ++n) {
      const int r = 8 * n + lrow;
      dma16(ad, cok && r < j.a.rows ? (uint32_t)r * ald + k0 : OUT, 0, base + NT * 2048 + SN * 256 + n * 1024);
    }
#pragma unroll
    for (int n = 0; n < SM; ++n) {
      const int x = 64 * n + lane, sl = x / TM, r = x - sl * TM;
      const bool ok = sl < 2 && 2 * u + sl < nslices && r < j.a.rows;
      dma4(as, ok ? (uint32_t)(2 * u + sl) * as4 + ((uint32_t)j.a.srow0 + (uint32_t)r) * 4u : OUT, 0,
           base + (NT + MT) * 2048 + SN * 256 + n * 256);
    }
  };
  v4f acc[MT][NT];
#pragma unroll
  for (int m = 0; m < MT; ++m)
#pragma unroll
    for (int n = 0; n < NT; ++n) acc[m][n] = v4f{0.0f, 0.0f, 0.0f, 0.0f};
  const int nu = __builtin_amdgcn_readfirstlane(((nblk + 7) / 8 - wave + WAVES - 1) / WAVES);  // the wave's units
#pragma unroll
  for (int i = 0; i < D; ++i) issue(i);
  for (int i = 0; i < nu; ++i) {
    wait_loads<(D - 1) * LOADS>();
    const uint8_t* pb = ring + (i % D) * UNIT;
    const uint8_t* pa = pb + NT * 2048 + SN * 256;
    const uint8_t *psb = pb + NT * 2048, *psa = pa + MT * 2048;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int at = ((4 * h + q) ^ (r16 & 7)) << 4;
      v8i a[MT], b[NT];
      int sa[MT], sb[NT];
#pragma unroll
      for (int n = 0; n < NT; ++n) {
        const v4i w = *reinterpret_cast<const v4i*>(pb + (16 * n + r16) * 128 + at);
        b[n] = v8i{w[0], w[1], w[2], w[3], 0, 0, 0, 0};
        sb[n] = psb[(h * TN + 16 * n + r16) * 4 + q];
      }
#pragma unroll
      for (int m = 0; m < MT; ++m) {
        const v4i w = *reinterpret_cast<const v4i*>(pa + (16 * m + r16) * 128 + at);
        a[m] = v8i{w[0], w[1], w[2], w[3], 0, 0, 0, 0};
        sa[m] = psa[(h * TM + 16 * m + r16) * 4 + q];
      }
#pragma unroll
      for (int m = 0; m < MT; ++m)
#pragma unroll
        for (int n = 0; n < NT; ++n)
          acc[m][n] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(b[n], a[m], acc[m][n], 4, 4, 0, sb[n], 0, sa[m]);
    }
    // the slot's reads are done (the MFMAs have their operands): refill it
    asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
    issue(i + D);
  }
  wait_loads<0>();
  __syncthreads();
  float(*part)[TM][PITCH] = reinterpret_cast<float(*)[TM][PITCH]>(smem);
  // every path out of the loop waits the last MFMAs out before the accumulators are read
  __builtin_amdgcn_sched_barrier(0);
  mfma_drain();
  __builtin_amdgcn_sched_barrier(0);
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

// ---------------------------------------------------------------------------------- large tile
//
// 256 x 256 output tile per workgroup, 4 waves of 128 x 128 (4 x 4 fragments of 32 x 32, 256 FP32
// accumulators per lane in AGPRs) on V_MFMA_SCALE_F32_32X32X64_F8F6F4, which issues faster than the
// 16 x 16 x 128 form (8.4 against 6.3 PFLOP/s in a loop without loads).  A K step is 256 elements: 128
// bytes a row, as in the MXFP8 kernel, whose direct-to-LDS loads and two stages it shares.  One 16-byte
// chunk is one scale block; chunk c of row r is stored at c ^ ((r >> 1) & 7), which keeps the 32-row
// fragment reads free of bank conflicts (with the MXFP8 kernel's r & 7, made for 16-row fragments, the
// conflicts counted were 0.47 of the LDS cycles).
//
// K order inside a step: lane half h = l / 32 takes chunks 4 h .. 4 h + 3, one per 64-wide MFMA
// (substep), the same for both operands, so its four block scales are the dword of K slice h that the
// K-step grouped layout keeps together, and each MFMA selects its byte.
//
// The loop is rotated: a substep's fragments are read from LDS behind the MFMAs of the one before, and
// the step's barrier stands before its last substep, whose fragments are in registers by then.  Behind
// the MFMAs of that substep the next step's first fragments are read and the loads of the step after it
// begin, so neither the LDS reads nor the barrier leave the matrix cores without work.
//
// What bounds it, in cycles of a CU (counted): 8192^3 takes 444,000 whatever the codes, of which the MFMAs are 262,000
// (2048 of a K step, 59%).  16 x 2048 x 4096 x 4096, the same K steps in eight tiles a CU instead of four, takes
// 514,000: a tile's start and end cost 17,600 cycles, 16% of 8192^3 and 27% of it.  The rest, 25%, is inside the K
// loop, 870 cycles of a step: its 68 KiB then come at 24 bytes per cycle and CU, and a kernel that only loads tiles in
// this order reached 21.  The time is those cycles at the clock the data leave: 208-213 us with every code equal
// (2.25 GHz), 258-299 us with random codes (1.8 GHz and less, lowest on a card that has been busy longer).
// Two workgroups per CU on 128 x 256 tiles, whose starts and ends overlap, need 1.5 times the operand loads per product
// and took 321 us where this kernel took 267 in the same run (8192^3).
constexpr int F4_KSTEP = 256;
constexpr int F4_ROWB = F4_KSTEP / 2;
constexpr int F4_DATA = BM2 * F4_ROWB;              // per operand and stage
constexpr int F4_SC = BM2 * 8;                       // scale bytes per operand and stage: [K slice][row] dwords
constexpr int F4_STAGE = 2 * (F4_DATA + F4_SC);      // A data, B data, A scales, B scales

// acc += B . A^T for one 64-wide substep; the scale of each operand is byte KK of its dword
template <int KK>
__device__ __forceinline__ void mfma_scale_fp4(v16f& acc, const v4i& b, const v4i& a, uint32_t sb, uint32_t sa) {
  if constexpr (KK == 0)
    asm volatile("v_mfma_scale_f32_32x32x64_f8f6f4 %0, %1, %2, %0, %3, %4 op_sel_hi:[0,0,0] cbsz:4 blgp:4"
                 : "+a"(acc) : "v"(b), "v"(a), "v"(sb), "v"(sa));
  else if constexpr (KK == 1)
    asm volatile("v_mfma_scale_f32_32x32x64_f8f6f4 %0, %1, %2, %0, %3, %4 op_sel:[1,1,0] op_sel_hi:[0,0,0] cbsz:4 blgp:4"
                 : "+a"(acc) : "v"(b), "v"(a), "v"(sb), "v"(sa));
  else if constexpr (KK == 2)
    asm volatile("v_mfma_scale_f32_32x32x64_f8f6f4 %0, %1, %2, %0, %3, %4 op_sel_hi:[1,1,0] cbsz:4 blgp:4"
                 : "+a"(acc) : "v"(b), "v"(a), "v"(sb), "v"(sa));
  else
    asm volatile("v_mfma_scale_f32_32x32x64_f8f6f4 %0, %1, %2, %0, %3, %4 op_sel:[1,1,0] op_sel_hi:[1,1,0] cbsz:4 blgp:4"
                 : "+a"(acc) : "v"(b), "v"(a), "v"(sb), "v"(sa));
}

// Epilogue: lane (r32, h32) of wave (wm, wn) holds, for fragment (fm, fn) and register group g, output row
// 128 wm + 32 fm + r32 and the four columns 128 wn + 32 fn + 8 g + 4 h32 .. + 3.  Stored from there, an
// instruction would write 32 bytes of each of 32 rows; 32 rows at a time go through the wave's part of LDS
// instead (free by then) and leave it as whole 256-byte (FP32: 512-byte) row pieces, non-temporal: the
// outputs of the tiles in flight fill the L2, and the operands are read again.  16 x 2048 x 4096 x 4096, in one run:
// 288 us (331 from the fragments, 317 through LDS with plain stores); its weight gradient in FP32 407 us (560, 470).
// (The same launches in a traced run of 40 in a row: 332 us at the median, 302 at least; the gradient 435 and 408,
// accumulating 637 and 602.)
template <bool F32>
__device__ __forceinline__ void epilogue_fp4(const TileJob& j, v16f (&acc)[4][4], const uint2* bias_lds, uint8_t* buf,
                                             bool accumulate, int wm, int wn, int lane) {
  constexpr int STORE_NT = 2;  // cache policy of the buffer store
  constexpr int ES = F32 ? 4 : 2, LPR = 128 * ES / 16, RPI = 64 / LPR;  // lanes per row, rows per instruction
  constexpr int PITCH = 128 * ES + 16;  // the padding spreads the rows over the banks
  const int r32 = lane & 31, h32 = lane >> 5, lr = lane / LPR, lc = lane % LPR;
  const uint32_t ldb = (uint32_t)j.ldc * ES;
  // columns past the tile's end: an offset past every record count
  const uint32_t vo = wn * 128 * ES + 16 * lc < j.b.rows * ES ? (uint32_t)lr * ldb + 16u * (uint32_t)lc : 0x80000000u;
#pragma unroll
  for (int fm = 0; fm < 4; ++fm) {
    const int row0 = wm * 128 + fm * 32;
    if (row0 >= j.a.rows) continue;
#pragma unroll
    for (int fn = 0; fn < 4; ++fn) {
#pragma unroll
      for (int g = 0; g < 4; ++g) {
        float v[4];
#pragma unroll
        for (int t = 0; t < 4; ++t) v[t] = acc[fm][fn][4 * g + t];
        const uint2 bw = bias_lds[(wn * 128 + fn * 32 + 8 * g + 4 * h32) >> 2];
        v[0] += bf16lo(bw.x); v[1] += bf16hi(bw.x); v[2] += bf16lo(bw.y); v[3] += bf16hi(bw.y);
        uint8_t* p = buf + r32 * PITCH + ES * (fn * 32 + 8 * g + 4 * h32);
        if constexpr (F32) *reinterpret_cast<float4*>(p) = make_float4(v[0], v[1], v[2], v[3]);
        else *reinterpret_cast<uint2*>(p) = make_uint2(bf16x2(v[0], v[1]), bf16x2(v[2], v[3]));
      }
    }
    // a wave's LDS accesses execute in order; this keeps the compiler's order
    asm volatile("" ::: "memory");
    const int64_t at = (j.crow0 + row0) * j.ldc + j.ccol0 + wn * 128;
    void* base = F32 ? static_cast<void*>(j.c32 + at) : static_cast<void*>(j.c16 + at);
    const int64_t bytes = (int64_t)std::min(j.a.rows - row0, 32) * j.ldc * ES;
    const __amdgpu_buffer_rsrc_t out = __builtin_amdgcn_make_buffer_rsrc(base, 0, (int)std::min<int64_t>(bytes, 0x7fffffff), RSRC_WORD3);
    constexpr int BATCH = 8;
#pragma unroll
    for (int i0 = 0; i0 < 32 / RPI; i0 += BATCH) {
      v4u w[BATCH];
#pragma unroll
      for (int i = 0; i < BATCH; ++i) w[i] = *reinterpret_cast<const v4u*>(buf + (RPI * (i0 + i) + lr) * PITCH + 16 * lc);
      if (F32 && accumulate) {
        v4u o[BATCH];
#pragma unroll
        for (int i = 0; i < BATCH; ++i) o[i] = __builtin_amdgcn_raw_buffer_load_b128(out, (int)(vo + (uint32_t)(RPI * (i0 + i)) * ldb), 0, 0);
#pragma unroll
        for (int i = 0; i < BATCH; ++i)
#pragma unroll
          for (int t = 0; t < 4; ++t) w[i][t] = __float_as_uint(__uint_as_float(w[i][t]) + __uint_as_float(o[i][t]));
      }
#pragma unroll
      for (int i = 0; i < BATCH; ++i) {
        __builtin_amdgcn_raw_buffer_store_b128(w[i], out, (int)(vo + (uint32_t)(RPI * (i0 + i)) * ldb), 0, STORE_NT);
        asm volatile("s_nop 1" ::"v"(w[i]));
      }
    }
    asm volatile("" ::: "memory");
  }
}

template <bool F32>
__global__ __launch_bounds__(256) __attribute__((amdgpu_waves_per_eu(1, 1)))
void gemm_mxfp4_256_kernel(GemmArgs ga, GemmTable tt) {
  __shared__ __attribute__((aligned(1024))) uint8_t smem[2 * F4_STAGE];
  __shared__ __attribute__((aligned(16))) uint2 bias_lds[BN2 / 4];
  int tile;
  TileJob j;
  if (tt.dev) {
    if (!schedule_tile(*tt.dev, blockIdx.x, &tile)) return;
    j = make_job<MGS_FMT_MXFP4, BM2, BN2>(ga, *tt.dev, tile);
  } else {
    if (!schedule_tile(tt, blockIdx.x, &tile)) return;
    j = make_job<MGS_FMT_MXFP4, BM2, BN2>(ga, tt, tile);
  }
  if (j.k == 0) {
    write_zero_tile<BM2, BN2>(j, ga);
    return;
  }
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int wm = wave >> 1, wn = wave & 1;
  const int r32 = lane & 31, h32 = lane >> 5;
  const TileDma d = tile_dma(j, wave, lane);
  const uint32_t vs = (uint32_t)((wave * 64 + lane) * 4);
  // lane offset of the loads of 8-row groups n (even, odd): row 64 wave + 8 n + lane / 8, the chunk that
  // belongs at position lane % 8
  const int lrow = lane >> 3;
  const uint32_t lsw = (uint32_t)(((lane & 7) ^ (lrow >> 1)) << 4);
  const uint32_t va0 = (uint32_t)((wave * 64 + lrow) * j.a.ld), vb0 = (uint32_t)((wave * 64 + lrow) * j.b.ld);
  const uint32_t voa[2] = {va0 + lsw, va0 + (lsw ^ 64u)}, vob[2] = {vb0 + lsw, vb0 + (lsw ^ 64u)};

  // load instruction n of step st into stage `stg`: 0..7 B rows, 8..15 A rows (8 rows x 128 bytes each),
  // 16..19 the scale dwords of the wave's 64 rows (A and B, two K slices).  Rows and steps past the end
  // read what follows or zeros: those outputs are not stored, and a partial last step is masked.
  constexpr int NLOADS = 20;
  auto issue_one = [&](int st, uint8_t* stg, int n) {
    const uint32_t base = lds_addr(stg) + wave * 8 * 1024, k0 = (uint32_t)st * F4_ROWB;
    if (n < 8) {
      dma16(d.bd, vob[n & 1], n * d.b_ld8 + k0, base + F4_DATA + n * 1024);
    } else if (n < 16) {
      dma16(d.ad, voa[n & 1], (n - 8) * d.a_ld8 + k0, base + (n - 8) * 1024);
    } else {
      const uint32_t sl = (uint32_t)n & 1u, sc = lds_addr(stg) + 2 * F4_DATA + sl * (BM2 * 4) + wave * 256;
      if (n < 18) dma4(d.bs, vs, (2u * (uint32_t)st + sl) * d.b_s4 + d.b_sr, sc + F4_SC);
      else dma4(d.as, vs, (2u * (uint32_t)st + sl) * d.a_s4 + d.a_sr, sc);
    }
  };

  v16f acc[4][4];
  // fragment f of the wave's 128 rows: row 128 w + 32 f + r32; rows 32 f apart share the chunk swizzle
  const uint32_t ra = (uint32_t)(wm * 128 + r32) * F4_ROWB, rb = (uint32_t)(wn * 128 + r32) * F4_ROWB + F4_DATA;
  const uint32_t sa0 = 2 * F4_DATA + h32 * (BM2 * 4) + (wm * 128 + r32) * 4, sb0 = sa0 + F4_SC + (wn - wm) * 512;
  auto frag = [&](const uint8_t* stg, uint32_t row, int f, int kk) {
    return *reinterpret_cast<const v4i*>(stg + row + f * 32 * F4_ROWB + (((4 * h32 + kk) ^ ((r32 >> 1) & 7)) << 4));
  };
  v4i fa[2][4], fb[2][4];          // fragments of the even and odd substeps
  uint32_t sa[4], sb[4], na[4], nb[4];  // scale dwords of this step and the next
  // read i (0..7) of substep kk: B fragments, then A; read 8..15 the step's scales
  auto read_one = [&](const uint8_t* stg, int kk, int buf, int i) {
    if (i < 4) fb[buf][i] = frag(stg, rb, i, kk);
    else if (i < 8) fa[buf][i - 4] = frag(stg, ra, i - 4, kk);
    else if (i < 12) nb[i - 8] = *reinterpret_cast<const uint32_t*>(stg + sb0 + (i - 8) * 128);
    else na[i - 12] = *reinterpret_cast<const uint32_t*>(stg + sa0 + (i - 12) * 128);
  };

  const int nsteps = __builtin_amdgcn_readfirstlane((int)((j.k + F4_KSTEP - 1) / F4_KSTEP));
  const int last_rem = (int)(j.k - (int64_t)(nsteps - 1) * F4_KSTEP);

  // the 16 MFMAs of substep KK from fragment buffer KK % 2, `behind(m)` after the m-th
  auto substep = [&](auto kk, auto&& behind) {
    constexpr int KK = decltype(kk)::value, B = KK & 1;
#pragma unroll
    for (int fm = 0; fm < 4; ++fm)
#pragma unroll
      for (int fn = 0; fn < 4; ++fn) {
        mfma_scale_fp4<KK>(acc[fm][fn], fb[B][fn], fa[B][fm], sb[fn], sa[fm]);
        behind(4 * fm + fn);
        __builtin_amdgcn_sched_barrier(0);
      }
  };
  // K elements past the end of the reduction: zero codes with the scale code 0
  auto mask = [&](int kk) {
    const int left = last_rem - 128 * h32;                // the lane's part of the step
    const bool ok = 32 * kk < left;
#pragma unroll
    for (int f = 0; f < 4; ++f) {
#pragma unroll
      for (int t = 0; t < 4; ++t) {
        fa[kk & 1][f][t] = ok ? fa[kk & 1][f][t] : 0;
        fb[kk & 1][f][t] = ok ? fb[kk & 1][f][t] : 0;
      }
      asm volatile("" : "+v"(fa[kk & 1][f]), "+v"(fb[kk & 1][f]));
      if (kk == 0) {
        const uint32_t m = left >= 128 ? 0xffffffffu : left <= 0 ? 0u : (1u << (left >> 2)) - 1u;  // 8 bits per 32 elements
        sa[f] &= m;
        sb[f] &= m;
        asm volatile("" : "+v"(sa[f]), "+v"(sb[f]));
      }
    }
    __builtin_amdgcn_sched_barrier(0);
    mfma_valu_gap();
    __builtin_amdgcn_sched_barrier(0);
  };
  constexpr std::integral_constant<int, 0> K0{};
  constexpr std::integral_constant<int, 1> K1{};
  constexpr std::integral_constant<int, 2> K2{};
  constexpr std::integral_constant<int, 3> K3{};
  // One K step.  The loads of step st + 1 (their first LEAD were issued in the step before) go out one per
  // PACE MFMAs.
  constexpr int PACE = 2, LEAD = 16 / PACE;
  auto step = [&](auto tail_tag, int st) {
    constexpr bool TAIL = decltype(tail_tag)::value;
    uint8_t* stg = smem + (st & 1) * F4_STAGE;
    uint8_t* nxt = smem + ((st + 1) & 1) * F4_STAGE;
    const bool more = !TAIL && st + 1 < nsteps, more2 = !TAIL && st + 2 < nsteps;
    auto feed = [&](int m) {  // m-th MFMA of the step's first three substeps (step 1 was loaded with step 0)
      if (more && st > 0 && m % PACE == PACE - 1 && LEAD + m / PACE < NLOADS) issue_one(st + 1, nxt, LEAD + m / PACE);
    };
#pragma unroll
    for (int f = 0; f < 4; ++f) {
      sa[f] = na[f];
      sb[f] = nb[f];
      asm volatile("" : "+v"(sa[f]), "+v"(sb[f]));
    }
    __builtin_amdgcn_sched_barrier(0);
    mfma_valu_gap();
    __builtin_amdgcn_sched_barrier(0);
    if (TAIL) mask(0);
    substep(K0, [&](int m) { if (m < 8) read_one(stg, 1, 1, m); feed(m); });
    if (TAIL) mask(1);
    substep(K1, [&](int m) { if (m < 8) read_one(stg, 2, 0, m); feed(16 + m); });
    if (TAIL) mask(2);
    substep(K2, [&](int m) { if (m < 8) read_one(stg, 3, 1, m); feed(32 + m); });
    if (TAIL) mask(3);
    // from here on the other stage is loaded and this one read by every wave
    __builtin_amdgcn_s_waitcnt(0);
    __syncthreads();
    substep(K3, [&](int m) {
      if (more) {
        if (m < 8) read_one(nxt, 0, 0, m);
        else if (m < 12) { read_one(nxt, 0, 0, 2 * m - 8); read_one(nxt, 0, 0, 2 * m - 7); }
      }
      if (more2 && m % PACE == PACE - 1) issue_one(st + 2, stg, m / PACE);
    });
    // the tile's last MFMAs are waited out on each path (accumulator copies may follow the join)
    if (!more) {
      __builtin_amdgcn_sched_barrier(0);
      mfma_drain();
      __builtin_amdgcn_sched_barrier(0);
    }
  };

  // (without a bias zeros)
  if (wave < 2) dma4(d.bias, d.has_bias ? (uint32_t)(wave * 256 + lane * 4) : 0x80000000u, 0, lds_addr(bias_lds) + wave * 256);
#pragma unroll
  for (int n = 0; n < NLOADS; ++n) issue_one(0, smem, n);
  if (nsteps > 1)
#pragma unroll
    for (int n = 0; n < NLOADS; ++n) issue_one(1, smem + F4_STAGE, n);
  // (the accumulators are cleared while the loads are under way)
#pragma unroll
  for (int fm = 0; fm < 4; ++fm)
#pragma unroll
    for (int fn = 0; fn < 4; ++fn) acc[fm][fn] = v16f{};
  __builtin_amdgcn_sched_barrier(0);
  mfma_valu_gap();
  __builtin_amdgcn_sched_barrier(0);
  if (nsteps > 1) wait_loads<NLOADS>();
  else wait_loads<0>();
  __syncthreads();
#pragma unroll
  for (int i = 0; i < 16; ++i) read_one(smem, 0, 0, i);
  const bool tail = last_rem < F4_KSTEP;
  const int full = tail ? nsteps - 1 : nsteps;
  for (int st = 0; st < full; ++st) step(std::false_type{}, st);
  if (tail) step(std::true_type{}, nsteps - 1);
  __builtin_amdgcn_sched_barrier(0);
  mfma_drain();
  __builtin_amdgcn_sched_barrier(0);
  epilogue_fp4<F32>(j, acc, bias_lds, smem + wave * (2 * F4_STAGE / 4), ga.accumulate != 0, wm, wn, lane);
}
