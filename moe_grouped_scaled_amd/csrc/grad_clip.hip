// The global 2-norm of many gradients, and the gradients scaled down to a largest norm.
//   norm = sqrt(sum of all squares);  out = g * min(1, max_norm / (norm + eps))
//
// Squares and their sums are FP64 (a BF16 or FP32 gradient's square can overflow or vanish in FP32, and the sum has up to
// billions of terms); the FP64 multiply-adds run at half the FP32 rate here, far above what memory delivers.
// A tensor is cut into chunks, each with one partial sum in the workspace; up to FEW of them every workgroup of the
// scaling launch adds them up itself, in the same fixed order; more are added by a launch of one workgroup between
// the two.  No result depends on timing.  The tensors' addresses travel in the kernel arguments, TENSORS of them a
// launch; where there are more, such launches first put them into the workspace, so that the norm and the scaling
// are one launch each (400 tensors, 1.2 GB: in four launches each they took 219 and 577 us).
// Bound by memory: those 400 tensors take 199 us for the norm (6.1 TB/s) and 478 us for the scaling (5.1 TB/s read and
// written), 3.2 GB of FP32 gradients into BF16 518 and 905 us; 12 tensors of 300000 elements 3.8 and 4.3 us.
#include <algorithm>
#include <cmath>
#include <new>
#include <vector>

#include "mgs_device.h"
#include "mgs_span.h"

namespace mgs {
namespace {

constexpr int TENSORS = 120;     // a launch: 3.8 KiB of kernel arguments
constexpr int UNIT = 8;          // elements that a thread takes at a time
constexpr int UNITS = 4;         // units of a thread under way

struct Entry {
  const void* in;
  void* out;
  int64_t n;
  int32_t first;                 // chunks before this tensor
  int32_t types;                 // bit 0: the input is FP32, bit 1: the output is
};
struct Batch {
  Entry e[TENSORS];
  const Entry* dev;              // all entries in the workspace; NULL: they are e
  int32_t count, chunk;          // tensors; elements of a chunk, a multiple of 2048
};

// Elements of a chunk: about 8192 chunks in all, at least 2048 elements (one round of a workgroup) and at most 2^20.
int64_t chunk_of(int64_t total) {
  const int64_t c = (total / 8192 + 2047) / 2048 * 2048;
  return c < 2048 ? 2048 : c > (1 << 20) ? (1 << 20) : c;
}
constexpr int64_t FEW = 1024;    // partial sums that a workgroup adds up by itself

typedef unsigned int v4u __attribute__((ext_vector_type(4)));

__device__ __forceinline__ double wave_sum(double v) {
#pragma unroll
  for (int o = 32; o; o >>= 1) v += __shfl_xor(v, o);
  return v;
}

// The workgroup's sum, in all of its threads.
__device__ __forceinline__ double block_sum(double v) {
  __shared__ double s[4];
  v = wave_sum(v);
  if ((threadIdx.x & 63) == 0) s[threadIdx.x >> 6] = v;
  __syncthreads();
  v = ((s[0] + s[1]) + s[2]) + s[3];
  __syncthreads();
  return v;
}

// The tensor of a chunk.  DEV: the entries are in the workspace (a template, since a choice between the two at run
// time has the compiler copy the arguments to scratch).
template <bool DEV>
__device__ __forceinline__ Entry entry_of(const Batch& b, int chunk) {
  if constexpr (DEV) {
    // the number of tensors that begin at or before the chunk, all compared at once
    int t = -1;
    for (int i0 = 0; i0 < b.count; i0 += 256) {
      const int i = i0 + (int)threadIdx.x;
      t += __syncthreads_count(i < b.count && b.dev[i].first <= chunk);
    }
    return b.dev[t];
  } else {
    int lo = 0, hi = b.count;
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if (b.e[mid].first <= chunk) lo = mid; else hi = mid;
    }
    return Entry{b.e[lo].in, b.e[lo].out, b.e[lo].n, b.e[lo].first, b.e[lo].types};
  }
}

__global__ __launch_bounds__(128) void table_kernel(Batch b, int n, Entry* __restrict__ out) {
  if ((int)threadIdx.x < n) out[threadIdx.x] = b.e[threadIdx.x];
}

// Eight elements from p on (16-byte aligned), or one.
template <bool F32>
struct Eight {
  v4u w[F32 ? 2 : 1];
  __device__ __forceinline__ void load(const uint8_t* p) {
    w[0] = *reinterpret_cast<const v4u*>(p);
    if constexpr (F32) w[1] = *reinterpret_cast<const v4u*>(p + 16);
  }
  __device__ __forceinline__ float get(int i) const {
    if constexpr (F32) return __uint_as_float(w[i >> 2][i & 3]);
    else return i & 1 ? bf16hi(w[0][i >> 1]) : bf16lo(w[0][i >> 1]);
  }
};
template <bool F32>
__device__ __forceinline__ float one_of(const void* p, int64_t i) {
  if constexpr (F32) return static_cast<const float*>(p)[i];
  else return bf16lo(static_cast<const uint16_t*>(p)[i]);
}

// Elements before the first 16-byte boundary at or behind element lo (at most `most`).
template <bool F32>
__device__ __forceinline__ int head_of(const void* p, int64_t lo, int64_t most) {
  constexpr int ES = F32 ? 4 : 2;
  return (int)min<int64_t>(most, ((16 - ((reinterpret_cast<uintptr_t>(p) + lo * ES) & 15)) & 15) / ES);
}

template <bool F32>
__device__ __forceinline__ double squares(const void* p, int64_t lo, int64_t hi) {
  constexpr int ES = F32 ? 4 : 2;
  const int head = head_of<F32>(p, lo, hi - lo);
  const int64_t units = (hi - lo - head) / UNIT, tail = lo + head + units * UNIT;
  double s = 0.0;
  auto add = [&](float v) { s = __builtin_fma((double)v, (double)v, s); };
  if ((int)threadIdx.x < head) add(one_of<F32>(p, lo + threadIdx.x));
  const uint8_t* base = static_cast<const uint8_t*>(p) + (lo + head) * ES;
  int64_t u = threadIdx.x;
  for (; u + (UNITS - 1) * 256 < units; u += UNITS * 256) {
    Eight<F32> e[UNITS];
#pragma unroll
    for (int i = 0; i < UNITS; ++i) e[i].load(base + (u + i * 256) * UNIT * ES);
#pragma unroll
    for (int i = 0; i < UNITS; ++i)
#pragma unroll
      for (int t = 0; t < UNIT; ++t) add(e[i].get(t));
  }
  for (; u < units; u += 256) {
    Eight<F32> e;
    e.load(base + u * UNIT * ES);
#pragma unroll
    for (int t = 0; t < UNIT; ++t) add(e.get(t));
  }
  if (tail + threadIdx.x < hi) add(one_of<F32>(p, tail + threadIdx.x));
  return s;
}

template <bool DEV>
__global__ __launch_bounds__(256) void norm_kernel(Batch b, double* __restrict__ part) {
  const Entry e = entry_of<DEV>(b, blockIdx.x);
  const int64_t lo = (int64_t)((int)blockIdx.x - e.first) * b.chunk, hi = min<int64_t>(e.n, lo + b.chunk);
  const double s = block_sum(e.types & 1 ? squares<true>(e.in, lo, hi) : squares<false>(e.in, lo, hi));
  if (threadIdx.x == 0) part[blockIdx.x] = s;
}

// The square root of the sum of `parts` partial sums.  All of a thread's loads go out before they are added.
__device__ __forceinline__ double total_norm(const double* part, int64_t parts) {
  double s = 0.0;
  int64_t i = threadIdx.x;
  for (; i + 3 * 256 < parts; i += 4 * 256) {
    const double a = part[i], b = part[i + 256], c = part[i + 512], d = part[i + 768];
    s = (((s + a) + b) + c) + d;
  }
  for (; i < parts; i += 256) s += part[i];
  return sqrt(block_sum(s));
}

// the norm, in FP32 for the caller and (nullable) in FP64 for the scaling launch
__global__ __launch_bounds__(256) void norm_total_kernel(const double* __restrict__ part, int64_t parts, float* __restrict__ norm,
                                                         double* __restrict__ wide) {
  const double v = total_norm(part, parts);
  if (threadIdx.x == 0) {
    *norm = (float)v;
    if (wide) *wide = v;
  }
}

template <bool F32>
__device__ __forceinline__ void put8(uint8_t* p, const float (&v)[UNIT]) {
  v4u w[2];
  if constexpr (F32) {
#pragma unroll
    for (int i = 0; i < 8; ++i) w[i >> 2][i & 3] = __float_as_uint(v[i]);
    __builtin_nontemporal_store(w[0], reinterpret_cast<v4u*>(p));
    __builtin_nontemporal_store(w[1], reinterpret_cast<v4u*>(p + 16));
    asm volatile("s_nop 1" ::"v"(w[0]), "v"(w[1]));  // (a wide store reads its data after it issues)
  } else {
    w[0] = v4u{bf16x2(v[0], v[1]), bf16x2(v[2], v[3]), bf16x2(v[4], v[5]), bf16x2(v[6], v[7])};
    __builtin_nontemporal_store(w[0], reinterpret_cast<v4u*>(p));
    asm volatile("s_nop 1" ::"v"(w[0]));
  }
}
template <bool F32>
__device__ __forceinline__ void put1(void* p, int64_t i, float v) {
  if constexpr (F32) static_cast<float*>(p)[i] = v;
  else static_cast<uint16_t*>(p)[i] = (uint16_t)bf16x2(v, 0.0f);
}

template <bool IN32, bool OUT32>
__device__ __forceinline__ void scaled(const void* in, void* out, int64_t lo, int64_t hi, float scale) {
  constexpr int IS = IN32 ? 4 : 2, OS = OUT32 ? 4 : 2;
  // Units start where both are 16-byte aligned.  Where that is nowhere (an input and an output at odd distances, or
  // of two types at odd places), elements go one by one.
  int head = head_of<IN32>(in, lo, hi - lo);
  constexpr int STEP = IN32 ? 4 : 8;
  auto fits = [&](int h) { return ((reinterpret_cast<uintptr_t>(out) + (lo + h) * OS) & 15) == 0; };
  if (!fits(head) && head + STEP < UNIT && fits(head + STEP)) head += STEP;
  if (!fits(head) || head > hi - lo) head = (int)(hi - lo);
  const int64_t units = (hi - lo - head) / UNIT, tail = lo + head + units * UNIT;
  for (int64_t i = lo + threadIdx.x; i < lo + head; i += 256) put1<OUT32>(out, i, one_of<IN32>(in, i) * scale);
  const uint8_t* src = static_cast<const uint8_t*>(in) + (lo + head) * IS;
  uint8_t* dst = static_cast<uint8_t*>(out) + (lo + head) * OS;
  auto put = [&](const Eight<IN32>& e, int64_t u) {
    float v[UNIT];
#pragma unroll
    for (int t = 0; t < UNIT; ++t) v[t] = e.get(t) * scale;
    put8<OUT32>(dst + u * UNIT * OS, v);
  };
  int64_t u = threadIdx.x;
  for (; u + (UNITS - 1) * 256 < units; u += UNITS * 256) {
    Eight<IN32> e[UNITS];
#pragma unroll
    for (int i = 0; i < UNITS; ++i) e[i].load(src + (u + i * 256) * UNIT * IS);
#pragma unroll
    for (int i = 0; i < UNITS; ++i) put(e[i], u + i * 256);
  }
  for (; u < units; u += 256) {
    Eight<IN32> e;
    e.load(src + u * UNIT * IS);
    put(e, u);
  }
  if (tail + threadIdx.x < hi) put1<OUT32>(out, tail + threadIdx.x, one_of<IN32>(in, tail + threadIdx.x) * scale);
}

// Chunks are taken from the last to the first: the norm's launch has just read them, and what of them is in the caches
// need not come from memory again.  `wide`: the norm; NULL: the `parts` partial sums are added here.
template <bool DEV>
__global__ __launch_bounds__(256) void scale_kernel(Batch b, const double* __restrict__ part, int64_t parts, const double* __restrict__ wide,
                                                    float max_norm, float eps, float* __restrict__ norm) {
  const double v = wide ? *wide : total_norm(part, parts);
  if (!wide && blockIdx.x == 0 && threadIdx.x == 0) *norm = (float)v;
  const double c = (double)max_norm / (v + (double)eps);
  const float scale = c >= 1.0 ? 1.0f : (float)c;  // NaN stays NaN
  const int chunk = gridDim.x - 1 - blockIdx.x;
  const Entry e = entry_of<DEV>(b, chunk);
  if (scale == 1.0f && e.in == e.out) return;  // in place, nothing to change
  const int64_t lo = (int64_t)(chunk - e.first) * b.chunk, hi = min<int64_t>(e.n, lo + b.chunk);
  switch (e.types) {
    case 0: scaled<false, false>(e.in, e.out, lo, hi, scale); break;
    case 1: scaled<true, false>(e.in, e.out, lo, hi, scale); break;
    case 2: scaled<false, true>(e.in, e.out, lo, hi, scale); break;
    default: scaled<true, true>(e.in, e.out, lo, hi, scale); break;
  }
}

int64_t chunks_of(int64_t n, int64_t chunk) { return (n + chunk - 1) / chunk; }

// What a call works on: chunks and their size, tensors that are not empty, workspace bytes (partial sums and the norm;
// then the entries, where they do not fit into one launch's arguments).
struct Plan {
  int64_t chunk, chunks, tensors, table_at, bytes;
};

int plan_of(int32_t count, const mgs_grad* grads, Plan* p) {
  if (count < 0) return fail(MGS_ERR_INVALID_ARG, "the number of tensors is negative");
  if (count > 0 && !grads) return fail(MGS_ERR_INVALID_ARG, "grads is NULL");
  int64_t total = 0;
  *p = Plan{};
  for (int32_t i = 0; i < count; ++i) {
    const mgs_grad& g = grads[i];
    if (g.numel < 0) return fail(MGS_ERR_SHAPE, "grads[%d].numel is negative", i);
    if (g.numel > 0 && !g.grad) return fail(MGS_ERR_INVALID_ARG, "grads[%d].grad is NULL", i);
    if ((g.grad_dtype != MGS_DTYPE_BF16 && g.grad_dtype != MGS_DTYPE_F32) ||
        (g.out_dtype != MGS_DTYPE_BF16 && g.out_dtype != MGS_DTYPE_F32))
      return fail(MGS_ERR_INVALID_ARG, "grads[%d] has an unknown dtype", i);
    const int is = g.grad_dtype == MGS_DTYPE_F32 ? 4 : 2, os = g.out_dtype == MGS_DTYPE_F32 ? 4 : 2;
    if (reinterpret_cast<uintptr_t>(g.grad) % is || reinterpret_cast<uintptr_t>(g.out) % os)
      return fail(MGS_ERR_INVALID_ARG, "grads[%d] is not aligned to its elements", i);
    if (g.numel > (int64_t)1 << 40) return fail(MGS_ERR_SHAPE, "grads[%d].numel is above 2^40", i);
    total = std::min<int64_t>(total + g.numel, (int64_t)1 << 60);
  }
  p->chunk = chunk_of(total);
  for (int32_t i = 0; i < count; ++i) {
    p->chunks += chunks_of(grads[i].numel, p->chunk);
    p->tensors += grads[i].numel > 0;
  }
  if (p->chunks > INT32_MAX / 256) return fail(MGS_ERR_SHAPE, "too many elements");
  p->table_at = 8 * (p->chunks + 1);
  p->bytes = p->table_at + (p->tensors > TENSORS ? p->tensors * (int64_t)sizeof(Entry) : 0);
  return MGS_OK;
}

// Outputs (scaled gradients, the norm, the workspace) must not overlap each other or a gradient, but for a gradient
// scaled in place: the ranges in address order, each against the furthest end before it.
int check_overlaps(int32_t count, const mgs_grad* grads, bool clip, const Range& norm, const Range& ws) {
  struct Span { uintptr_t lo, hi; bool out; };
  std::vector<Span> v;
  v.reserve(2 * (size_t)count + 2);
  auto add = [&](const void* p, int64_t bytes, bool out) {
    if (p && bytes > 0) v.push_back({reinterpret_cast<uintptr_t>(p), reinterpret_cast<uintptr_t>(p) + (uintptr_t)bytes, out});
  };
  add(norm.p, norm.bytes, true);
  add(ws.p, ws.bytes, true);
  for (int32_t i = 0; i < count; ++i) {
    const mgs_grad& g = grads[i];
    const int64_t in = (g.grad_dtype == MGS_DTYPE_F32 ? 4 : 2) * g.numel, out = (g.out_dtype == MGS_DTYPE_F32 ? 4 : 2) * g.numel;
    const bool in_place = clip && g.out == g.grad && g.out_dtype == g.grad_dtype;
    add(g.grad, in, in_place);
    if (clip && !in_place) add(g.out, out, true);
  }
  std::sort(v.begin(), v.end(), [](const Span& a, const Span& b) { return a.lo < b.lo; });
  uintptr_t all = 0, outs = 0;
  for (const Span& s : v) {
    if (s.lo < (s.out ? all : outs))
      return fail(MGS_ERR_INVALID_ARG, "an output must not be or overlap another tensor of the call (a gradient scaled in place is "
                  "given once, as its own output)");
    all = std::max(all, s.hi);
    if (s.out) outs = std::max(outs, s.hi);
  }
  return MGS_OK;
}

}  // namespace
}  // namespace mgs

using namespace mgs;

extern "C" {

int64_t mgs_grad_norm_workspace_bytes(int32_t count, const mgs_grad* grads) {
  Plan p;
  const int rc = plan_of(count, grads, &p);
  if (rc) return rc;
  ok();
  return p.bytes;
}

int mgs_grad_norm(int32_t count, const mgs_grad* grads, float* norm, void* workspace, int64_t workspace_bytes, int32_t clip,
                  float max_norm, float eps, void* stream) {
  Plan p;
  int rc = plan_of(count, grads, &p);
  if (rc) return rc;
  if (!norm) return fail(MGS_ERR_INVALID_ARG, "norm is NULL");
  if (!workspace || workspace_bytes < p.bytes)
    return fail(MGS_ERR_INVALID_ARG, "a workspace of %lld bytes is needed (got %lld%s)", (long long)p.bytes,
                (long long)workspace_bytes, workspace ? "" : ", NULL");
  const Range rn{"norm", norm, 4}, rw{"the workspace", workspace, p.bytes};
  if ((rc = check_aligned({rn}, 4)) || (rc = check_aligned({rw}, 8))) return rc;
  if (clip && !(max_norm >= 0.0f && std::isfinite(max_norm))) return fail(MGS_ERR_INVALID_ARG, "max_norm must be finite and not negative");
  if (clip && !(eps >= 0.0f && std::isfinite(eps))) return fail(MGS_ERR_INVALID_ARG, "eps must be finite and not negative");
  for (int32_t i = 0; clip && i < count; ++i)
    if (grads[i].numel > 0 && !grads[i].out) return fail(MGS_ERR_INVALID_ARG, "grads[%d].out is NULL", i);
  try {
    if ((rc = check_overlaps(count, grads, clip != 0, rn, rw))) return rc;
  } catch (const std::bad_alloc&) {
    return fail(MGS_ERR_INVALID_ARG, "no host memory to check %d tensors", count);
  }
  const hipStream_t st = static_cast<hipStream_t>(stream);
  double* part = static_cast<double*>(workspace);
  double* wide = part + p.chunks;
  Entry* table = reinterpret_cast<Entry*>(static_cast<uint8_t*>(workspace) + p.table_at);
  Batch b{};
  b.count = (int32_t)p.tensors;
  b.chunk = (int32_t)p.chunk;
  const bool in_table = p.tensors > TENSORS;
  int used = 0;
  int64_t done = 0, first = 0;
  for (int32_t i = 0; i < count; ++i) {
    const mgs_grad& g = grads[i];
    if (g.numel == 0) continue;
    b.e[used++] = Entry{g.grad, g.out, g.numel, (int32_t)first,
                        (g.grad_dtype == MGS_DTYPE_F32 ? 1 : 0) | (g.out_dtype == MGS_DTYPE_F32 ? 2 : 0)};
    first += chunks_of(g.numel, p.chunk);
    if (in_table && (used == TENSORS || done + used == p.tensors)) {
      hipLaunchKernelGGL(table_kernel, dim3(1), dim3(128), 0, st, b, used, table + done);
      done += used;
      used = 0;
    }
  }
  if (in_table) b.dev = table;
  const dim3 grid((unsigned)p.chunks), block(256);
  const bool total = !clip || p.chunks == 0 || p.chunks > FEW;
  if (p.chunks > 0) hipLaunchKernelGGL(in_table ? norm_kernel<true> : norm_kernel<false>, grid, block, 0, st, b, part);
  if (total) hipLaunchKernelGGL(norm_total_kernel, dim3(1), block, 0, st, part, p.chunks, norm, wide);
  if (clip && p.chunks > 0) hipLaunchKernelGGL(in_table ? scale_kernel<true> : scale_kernel<false>, grid, block, 0, st, b, part, p.chunks, total ? wide : nullptr, max_norm, eps, norm);
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess) return fail(MGS_ERR_HIP, "HIP launch error: %s", hipGetErrorString(e));
  return ok();
}

}  // extern "C"
