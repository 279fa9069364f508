// The global 2-norm of many gradients, and the gradients scaled down to a largest norm.
//   norm = sqrt(sum of all squares);  out = g * min(1, max_norm / (norm + eps))
//
// Squares and their sums are FP64 (a BF16 or FP32 gradient's square can overflow or vanish in FP32, and the sum has up to
// billions of terms); the FP64 multiply-adds run at half the FP32 rate here, far above what memory delivers.
// A tensor is cut into chunks of CHUNK elements, each with one partial sum in the workspace; every workgroup of the
// scaling launch adds the partial sums in the same fixed order, so the result does not depend on timing and there
// is no launch between the two.  The tensors' addresses travel in the kernel arguments, TENSORS of them a launch.
#include <algorithm>
#include <cmath>
#include <new>
#include <vector>

#include "mgs_device.h"
#include "mgs_span.h"

namespace mgs {
namespace {

constexpr int TENSORS = 128;     // a launch: 3.6 KiB of kernel arguments
constexpr int64_t CHUNK = 1 << 16;

struct Batch {
  const void* in[TENSORS];
  void* out[TENSORS];
  int64_t n[TENSORS];
  int32_t first[TENSORS + 1];    // chunks of the batch before tensor i
  uint8_t in_f32[TENSORS], out_f32[TENSORS];
};

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

__device__ __forceinline__ int tensor_of(const Batch& b, int count, int chunk) {
  int lo = 0, hi = count;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (b.first[mid] <= chunk) lo = mid; else hi = mid;
  }
  return lo;
}

// f(i, value) for the elements [lo, hi) of a tensor that are this thread's: 16-byte pieces where the address allows
template <bool F32, typename Fn>
__device__ __forceinline__ void squares(const void* p, int64_t lo, int64_t hi, Fn f) {
  constexpr int V = F32 ? 4 : 8;
  const uint8_t* base = static_cast<const uint8_t*>(p);
  // elements up to the first 16-byte boundary
  const uintptr_t at = reinterpret_cast<uintptr_t>(base) + lo * (F32 ? 4 : 2);
  const int64_t head = min<int64_t>(hi, lo + (int64_t)((16 - (at & 15)) & 15) / (F32 ? 4 : 2));
  const int64_t units = (hi - head) / V;
  auto one = [&](int64_t i) { f(F32 ? static_cast<const float*>(p)[i] : bf16lo(static_cast<const uint16_t*>(p)[i])); };
  for (int64_t i = lo + threadIdx.x; i < head; i += 256) one(i);
  for (int64_t u = threadIdx.x; u < units; u += 256) {
    const v4u w = *reinterpret_cast<const v4u*>(base + (head + u * V) * (F32 ? 4 : 2));
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      if constexpr (F32) f(__uint_as_float(w[e]));
      else {
        f(bf16lo(w[e]));
        f(bf16hi(w[e]));
      }
    }
  }
  for (int64_t i = head + units * V + threadIdx.x; i < hi; i += 256) one(i);
}

__global__ __launch_bounds__(256) void norm_kernel(Batch b, int count, double* __restrict__ part) {
  const int t = tensor_of(b, count, blockIdx.x);
  const int64_t lo = (int64_t)(blockIdx.x - b.first[t]) * CHUNK, hi = min<int64_t>(b.n[t], lo + CHUNK);
  double s = 0.0;
  auto add = [&](float v) { s = __builtin_fma((double)v, (double)v, s); };
  if (b.in_f32[t]) squares<true>(b.in[t], lo, hi, add);
  else squares<false>(b.in[t], lo, hi, add);
  s = block_sum(s);
  if (threadIdx.x == 0) part[blockIdx.x] = s;
}

// the norm from all partial sums
__device__ __forceinline__ double total_norm(const double* part, int64_t parts) {
  double s = 0.0;
  for (int64_t i = threadIdx.x; i < parts; i += 256) s += part[i];
  return sqrt(block_sum(s));
}

__global__ __launch_bounds__(256) void norm_total_kernel(const double* __restrict__ part, int64_t parts, float* __restrict__ norm) {
  const double v = total_norm(part, parts);
  if (threadIdx.x == 0) *norm = (float)v;
}

__global__ __launch_bounds__(256) void scale_kernel(Batch b, int count, const double* __restrict__ part, int64_t parts, float max_norm,
                                                    float eps, float* __restrict__ norm) {
  const double v = total_norm(part, parts);
  if (norm && blockIdx.x == 0 && threadIdx.x == 0) *norm = (float)v;
  const double c = (double)max_norm / (v + (double)eps);
  const float scale = c < 1.0 ? (float)c : c >= 1.0 ? 1.0f : (float)c;  // NaN stays NaN
  const int t = tensor_of(b, count, blockIdx.x);
  const bool in32 = b.in_f32[t], out32 = b.out_f32[t];
  if (scale == 1.0f && b.in[t] == b.out[t]) return;  // in place, nothing to change
  const int64_t lo = (int64_t)(blockIdx.x - b.first[t]) * CHUNK, hi = min<int64_t>(b.n[t], lo + CHUNK);
  for (int64_t i = lo + threadIdx.x; i < hi; i += 256) {
    const float g = in32 ? static_cast<const float*>(b.in[t])[i] : bf16lo(static_cast<const uint16_t*>(b.in[t])[i]);
    const float o = g * scale;
    if (out32) static_cast<float*>(b.out[t])[i] = o;
    else static_cast<uint16_t*>(b.out[t])[i] = (uint16_t)bf16x2(o, 0.0f);
  }
}

int64_t chunks_of(int64_t n) { return (n + CHUNK - 1) / CHUNK; }

int check_tensors(int32_t count, const mgs_grad* grads, int64_t* chunks) {
  if (count < 0) return fail(MGS_ERR_INVALID_ARG, "the number of tensors is negative");
  if (count > 0 && !grads) return fail(MGS_ERR_INVALID_ARG, "grads is NULL");
  *chunks = 0;
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
    *chunks += chunks_of(g.numel);
  }
  if (*chunks > INT32_MAX / 256) return fail(MGS_ERR_SHAPE, "too many elements");
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
  int64_t chunks = 0;
  const int rc = check_tensors(count, grads, &chunks);
  if (rc) return rc;
  ok();
  return 8 * chunks;
}

int mgs_grad_norm(int32_t count, const mgs_grad* grads, float* norm, void* workspace, int64_t workspace_bytes, int32_t clip,
                  float max_norm, float eps, void* stream) {
  int64_t chunks = 0;
  int rc = check_tensors(count, grads, &chunks);
  if (rc) return rc;
  if (!norm) return fail(MGS_ERR_INVALID_ARG, "norm is NULL");
  if (chunks > 0 && (!workspace || workspace_bytes < 8 * chunks))
    return fail(MGS_ERR_INVALID_ARG, "a workspace of %lld bytes is needed (got %lld%s)", (long long)(8 * chunks),
                (long long)workspace_bytes, workspace ? "" : ", NULL");
  const Range rn{"norm", norm, 4}, rw{"the workspace", workspace, 8 * chunks};
  if ((rc = check_aligned({rn}, 4)) || (rc = check_aligned({rw}, 8))) return rc;
  if ((rc = check_ranges({rn, rw}, {}))) return rc;
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
  // launches over the tensors, TENSORS of them at a time
  auto batches = [&](auto&& launch) {
    Batch b;
    int used = 0;
    int64_t done = 0;
    b.first[0] = 0;
    auto flush = [&]() {
      if (used) launch(b, used, done);
      if (used) done += b.first[used];
      used = 0;
    };
    for (int32_t i = 0; i < count; ++i) {
      if (grads[i].numel == 0) continue;
      b.in[used] = grads[i].grad;
      b.out[used] = grads[i].out;
      b.n[used] = grads[i].numel;
      b.in_f32[used] = grads[i].grad_dtype == MGS_DTYPE_F32;
      b.out_f32[used] = grads[i].out_dtype == MGS_DTYPE_F32;
      b.first[used + 1] = b.first[used] + (int32_t)chunks_of(grads[i].numel);
      if (++used == TENSORS) flush();
    }
    flush();
  };
  batches([&](const Batch& b, int used, int64_t done) {
    hipLaunchKernelGGL(norm_kernel, dim3((unsigned)b.first[used]), dim3(256), 0, st, b, used, part + done);
  });
  if (!clip || chunks == 0) {
    hipLaunchKernelGGL(norm_total_kernel, dim3(1), dim3(256), 0, st, part, chunks, norm);
  } else {
    batches([&](const Batch& b, int used, int64_t done) {
      hipLaunchKernelGGL(scale_kernel, dim3((unsigned)b.first[used]), dim3(256), 0, st, b, used, part, chunks, max_norm, eps,
                         done == 0 ? norm : nullptr);
    });
  }
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess) return fail(MGS_ERR_HIP, "HIP launch error: %s", hipGetErrorString(e));
  return ok();
}

}  // extern "C"
