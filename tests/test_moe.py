"""Router, dispatch and combine without a GPU: refusals of the C entry points and of the Python calls, the
workspace size, and the host validation under the address and undefined-behaviour sanitizers."""

import ctypes
import os
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
FAKE = 0x1000  # never dereferenced: every call below fails validation before any launch


def _lib():
    from moe_grouped_scaled_amd import _native as N
    return N, N.LIB


def _refused(code, rc, match):
    N, lib = _lib()
    assert rc == code, (rc, lib.mgs_last_error())
    assert match in lib.mgs_last_error().decode(), lib.mgs_last_error()


def test_route_refusals():
    N, lib = _lib()
    p = N.RouteParams(0, 1, 1.0)

    def fwd(params=p, t=4, e=8, k=2, x=FAKE, dt=0, ld=8, idx=FAKE, w=FAKE):
        return lib.mgs_moe_route(params, t, e, k, x, dt, ld, idx, w, None)

    _refused(-1, fwd(None), "params")
    _refused(-1, fwd(N.RouteParams(2, 1, 1.0)), "score")
    _refused(-1, fwd(N.RouteParams(0, 1, float("inf"))), "finite")
    _refused(-1, fwd(N.RouteParams(0, 1, float("nan"))), "finite")
    for e in (0, -1, 257):
        _refused(-1, fwd(e=e), "num_experts")
    for k in (0, 9, 17):
        _refused(-1, fwd(k=k), "topk")
    _refused(-1, fwd(e=64, k=17, ld=64), "topk")
    for t in (-1, 1 << 30, 1 << 62):
        _refused(-2, fwd(t=t), "tokens")
    _refused(-1, fwd(dt=2), "dtype")
    _refused(-2, fwd(ld=7), "row stride")
    _refused(-1, fwd(x=None), "logits")
    _refused(-1, fwd(idx=None), "expert_idx")
    _refused(-1, fwd(w=None), "weights")
    assert fwd(t=0, x=None, idx=None, w=None) == 0
    bwd = lambda **k: lib.mgs_moe_route_bwd(p, k.get("t", 4), 8, 2, FAKE, 1, 8, k.get("idx", FAKE), k.get("dw", FAKE), k.get("dl", FAKE), k.get("ldd", 8), None)
    _refused(-2, bwd(ldd=7), "dlogits")
    for name in ("idx", "dw", "dl"):
        _refused(-1, bwd(**{name: None}), "is NULL")
    assert bwd(t=0, idx=None, dw=None, dl=None) == 0


def test_dispatch_and_combine_refusals():
    N, lib = _lib()

    def dis(t=4, k=2, e=8, idx=FAKE, h=64, dt=0, x=FAKE, ldx=64, w=None, rows=FAKE, n=8, rw=None, row=FAKE, sp=FAKE,
            ws=FAKE, wb=1 << 20):
        return lib.mgs_moe_dispatch(t, k, e, idx, h, dt, x, ldx, w, rows, n, rw, row, sp, ws, wb, None)

    for k in (0, 17):
        _refused(-1, dis(k=k), "topk")
    for e in (0, 257):
        _refused(-1, dis(e=e), "num_experts")
    for t in (-1, 1 << 30, 1 << 62):
        _refused(-2, dis(t=t), "tokens")
    _refused(-1, dis(idx=None), "expert_idx")
    _refused(-1, dis(row=None), "row_of_slot")
    _refused(-1, dis(sp=None), "split_sizes")
    _refused(-1, dis(x=None), "together")
    _refused(-1, dis(rows=None), "together")
    _refused(-1, dis(w=FAKE), "together")
    _refused(-1, dis(rw=FAKE), "together")
    _refused(-2, dis(n=7), "rows has 7 rows")
    _refused(-2, dis(h=0, ldx=0), "hidden")
    _refused(-2, dis(ldx=63), "row stride")
    _refused(-1, dis(dt=5), "dtype")
    need = lib.mgs_moe_dispatch_workspace_bytes(4000, 2, 8)
    assert need > 0
    _refused(-1, dis(t=4000, n=8000, wb=need - 1), "workspace")
    _refused(-1, dis(t=4000, n=8000, ws=None), "workspace")
    for bad in ((4, 0, 8), (4, 17, 8), (4, 2, 0), (4, 2, 257), (-1, 2, 8), (1 << 40, 2, 8)):
        assert lib.mgs_moe_dispatch_workspace_bytes(*bad) < 0

    com = lambda t=4, k=2, h=64, dt=0, row=FAKE, n=8, r=FAKE, y=FAKE, ld=64: lib.mgs_moe_combine(t, k, h, dt, row, n, r, None, y, ld, None)
    _refused(-1, com(k=0), "topk")
    _refused(-2, com(t=1 << 40), "tokens")
    _refused(-2, com(h=(1 << 24) + 1, ld=1 << 25), "hidden")
    _refused(-2, com(ld=63), "row stride")
    _refused(-2, com(n=1 << 31), "num_rows")
    _refused(-2, com(n=-1), "num_rows")
    for name in ("row", "r", "y"):
        _refused(-1, com(**{name: None}), "NULL")
    assert com(t=0, row=None, r=None, y=None) == 0
    back = lambda g=None, dw=None: lib.mgs_moe_dispatch_bwd(4, 2, 64, 0, FAKE, 8, FAKE, g, FAKE, 64, dw, None)
    _refused(-1, back(g=FAKE), "together")
    _refused(-1, back(dw=FAKE), "together")
    cb = lambda t=4, row=FAKE, dy=FAKE, r=FAKE, d=FAKE, dw=FAKE, ld=64: lib.mgs_moe_combine_bwd(t, 2, 64, 0, row, 8, dy, ld, r, None, d, dw, None)
    _refused(-1, cb(row=None), "NULL")
    _refused(-1, cb(dy=None), "NULL")
    _refused(-1, cb(d=None, dw=None), "no output")
    _refused(-1, cb(r=None), "needs rows")
    _refused(-2, cb(ld=1), "row stride")
    assert cb(t=0, row=None, dy=None) == 0


def test_python_calls_check_their_tensors():
    import torch
    import moe_grouped_scaled_amd as M
    f = lambda *s, dt=torch.float32: torch.zeros(s, dtype=dt)
    with pytest.raises(ValueError, match="on a GPU"):
        M.moe_route(f(4, 8), 2)
    with pytest.raises(ValueError, match="type"):
        M.moe_route(f(4, 8, dt=torch.float16), 2)
    with pytest.raises(ValueError, match="dimensions"):
        M.moe_route(f(8), 2)
    with pytest.raises(ValueError, match="column stride"):
        M.moe_route(f(8, 4).t(), 2)
    with pytest.raises(ValueError, match="do not overlap"):
        M.moe_route(f(1, 8).expand(4, 8), 2)
    with pytest.raises(ValueError, match="contiguous"):
        M.moe_dispatch(f(2, 4, dt=torch.int32).t(), 8)
    with pytest.raises(ValueError, match="type"):
        M.moe_dispatch(f(4, 2, dt=torch.int64), 8)
    with pytest.raises(ValueError, match="must be a tensor"):
        M.moe_combine(None, f(8, 8))
    from moe_grouped_scaled_amd.expert_mlp import ExpertMLP
    w = torch.zeros(2, 64, 64, dtype=torch.bfloat16)
    layer = M.MoELayer(ExpertMLP("srelu", "mxfp8", w, w), 2)
    with pytest.raises(ValueError, match="without a forward"):
        layer.backward(f(4, 64))
    with pytest.raises(ValueError, match="type"):
        layer.forward(f(4, 64), f(4, 2))


DRIVER = r"""
#include <cstdint>
#include <cstdio>
#include <climits>
#include "mgs.h"
int main() {
  int bad = 0, n = 0;
  int32_t* I = reinterpret_cast<int32_t*>(0x1000);
  float* F = reinterpret_cast<float*>(0x1000);
  void* P = reinterpret_cast<void*>(0x1000);
  int64_t* L = reinterpret_cast<int64_t*>(0x1000);
  const mgs_route_params ok{MGS_SCORE_SOFTMAX, 1, 1.0f}, odd{7, 1, 1.0f};
  const int64_t sizes[] = {INT64_MIN, -1, INT32_MAX, (int64_t)1 << 31, INT64_MAX};
  const int32_t counts[] = {INT32_MIN, -1, 0, 17, 257, INT32_MAX};
  auto want = [&](int64_t rc) { ++n; bad += rc >= 0; };
  want(mgs_moe_route(nullptr, 4, 8, 2, P, 0, 8, I, F, nullptr));
  want(mgs_moe_route(&odd, 4, 8, 2, P, 0, 8, I, F, nullptr));
  for (int64_t s : sizes) {
    want(mgs_moe_route(&ok, s, 8, 2, P, 0, 8, I, F, nullptr));
    want(mgs_moe_route_bwd(&ok, s, 8, 2, P, 0, 8, I, F, P, 8, nullptr));
    want(mgs_moe_dispatch_workspace_bytes(s, 2, 8));
    want(mgs_moe_dispatch(s, 2, 8, I, 64, 0, P, 64, nullptr, P, 1 << 20, nullptr, I, L, P, 1 << 20, nullptr));
    want(mgs_moe_combine(s, 2, 64, 0, I, 8, P, nullptr, P, 64, nullptr));
    want(mgs_moe_combine_bwd(s, 2, 64, 0, I, 8, P, 64, P, nullptr, P, F, nullptr));
    want(mgs_moe_dispatch_bwd(s, 2, 64, 0, I, 8, P, nullptr, P, 64, nullptr, nullptr));
    if (s != INT32_MAX) {
      want(mgs_moe_combine(4, 2, s, 0, I, 8, P, nullptr, P, INT64_MAX, nullptr));
      want(mgs_moe_combine(4, 2, 64, 0, I, s, P, nullptr, P, 64, nullptr));
    }
    if (s < 0) {
      want(mgs_moe_route(&ok, 4, 8, 2, P, 0, s, I, F, nullptr));
      want(mgs_moe_dispatch(4, 2, 8, I, 64, 0, P, s, nullptr, P, 8, nullptr, I, L, P, 1 << 20, nullptr));
      want(mgs_moe_dispatch(4000, 2, 8, I, 64, 0, P, 64, nullptr, P, 8000, nullptr, I, L, P, s, nullptr));
    }
  }
  for (int32_t c : counts) {
    want(mgs_moe_route(&ok, 4, 8, c, P, 0, 8, I, F, nullptr));
    if (c != 17) want(mgs_moe_route(&ok, 4, c, 2, P, 0, 8, I, F, nullptr));
    if (c != 257 && c != 17) want(mgs_moe_dispatch_workspace_bytes(4, 2, c));
    want(mgs_moe_dispatch_workspace_bytes(4, c, 8));
  }
  std::printf("%d calls, %d accepted\n", n, bad);
  return bad != 0;
}
"""


@pytest.mark.skipif(not os.path.exists("/opt/rocm/llvm/bin/clang++"), reason="needs the ROCm toolchain")
def test_host_validation_is_clean_under_sanitizers(tmp_path):
    hipcc, clang = os.environ.get("HIPCC", "/opt/rocm/bin/hipcc"), "/opt/rocm/llvm/bin/clang++"
    csrc = os.path.join(ROOT, "moe_grouped_scaled_amd", "csrc")
    san = ["-Xarch_host", "-fsanitize=address", "-Xarch_host", "-fsanitize=undefined", "-Xarch_host", "-fno-sanitize-recover=all"]

    def run(cmd, **kw):
        res = subprocess.run(cmd, stdout=subprocess.PIPE, stderr=subprocess.STDOUT, text=True, **kw)
        assert res.returncode == 0, res.stdout
        return res.stdout

    objs = []
    for src in ("mgs_api.hip", "act_quant.hip", "gemm_mx.hip", "moe_route.hip"):
        objs.append(str(tmp_path / src.replace(".hip", ".o")))
        run([hipcc, "--offload-arch=gfx950", "-O1", "-std=c++17", "-fPIC", *san, "-Xclang", "-target-feature", "-Xclang",
             "-packed-fp32-ops", "-c", os.path.join(csrc, src), "-o", objs[-1]])
    drv = tmp_path / "driver.cpp"
    drv.write_text(DRIVER)
    run([clang, "-O1", "-std=c++17", "-fsanitize=address,undefined", "-fno-sanitize-recover=all", "-I", os.path.join(ROOT, "include"),
         "-c", str(drv), "-o", str(tmp_path / "driver.o")])
    exe = str(tmp_path / "driver")
    run([hipcc, "--offload-arch=gfx950", *san[:4], "-o", exe, str(tmp_path / "driver.o"), *objs, "-Wl,-rpath,/opt/rocm/lib"])
    out = run([exe], env=dict(os.environ, ASAN_OPTIONS="detect_leaks=0"), timeout=120)
    assert " 0 accepted" in out
