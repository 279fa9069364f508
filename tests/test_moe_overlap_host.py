"""The overlap check of the routing calls under the undefined-behaviour sanitizer: sizes at the ends of what a call takes,
and widths that a call without rows does not look at (host code of csrc/moe_route.hip alone, linked with the two error
functions it uses)."""

import os
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

DRIVER = r"""
#include <climits>
#include <cstdarg>
#include <cstdint>
#include <cstdio>
#include <cstring>
#include <initializer_list>
#include "mgs.h"
static char msg[512];
namespace mgs {
int fail(int code, const char* fmt, ...) {
  va_list ap;
  va_start(ap, fmt);
  std::vsnprintf(msg, sizeof msg, fmt, ap);
  va_end(ap);
  return code;
}
int ok() { return 0; }
}
template <typename T> T* at(uintptr_t a) { return reinterpret_cast<T*>(a); }
int main() {
  int bad = 0;
  auto want = [&](int rc) {
    if (rc != MGS_ERR_INVALID_ARG || !std::strstr(msg, "must not be")) { ++bad; std::printf("%d %s\n", rc, msg); }
    msg[0] = 0;
  };
  // no rows: hidden and the stride are not looked at
  for (int64_t h : {INT64_MAX, INT64_MIN, (int64_t)-1, (int64_t)0})
    want(mgs_moe_dispatch(1 << 20, 16, 256, at<int32_t>(0x1000), h, 1, nullptr, h, nullptr, nullptr, h, nullptr, at<int32_t>(0x1000),
                          at<int64_t>(0x2000), at<void>(0x900000000), 1 << 30, nullptr));
  // the widest rows and the most of them
  const int64_t w = (int64_t)1 << 24, n = INT32_MAX;
  want(mgs_moe_combine(1 << 20, 16, w, 1, at<int32_t>(1ull << 62), n, at<void>(0x1000), nullptr, at<void>(0x2000), w, nullptr));
  want(mgs_moe_combine_bwd(1 << 20, 16, w, 1, at<int32_t>(1ull << 62), n, at<void>(0x2000), INT64_MAX, nullptr, at<float>(1ull << 61),
                           at<void>(0x1000), nullptr, nullptr));
  std::printf("%d wrong\n", bad);
  return bad != 0;
}
"""


@pytest.mark.skipif(not os.path.exists("/opt/rocm/llvm/bin/clang++"), reason="needs the ROCm toolchain")
def test_overlap_check_is_defined_for_every_size(tmp_path):
    from moe_grouped_scaled_amd.build import HIPCC
    san = ["-Xarch_host", "-fsanitize=undefined", "-Xarch_host", "-fno-sanitize-recover=all"]

    def run(cmd):
        res = subprocess.run(cmd, stdout=subprocess.PIPE, stderr=subprocess.STDOUT, text=True, timeout=300)
        assert res.returncode == 0, res.stdout
        return res.stdout

    obj, drv, exe = str(tmp_path / "moe_route.o"), tmp_path / "driver.cpp", str(tmp_path / "driver")
    run([HIPCC, "--offload-arch=gfx950", "-O1", "-std=c++17", "-fPIC", *san, "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops",
         "-c", os.path.join(ROOT, "moe_grouped_scaled_amd", "csrc", "moe_route.hip"), "-o", obj])
    drv.write_text(DRIVER)
    run(["/opt/rocm/llvm/bin/clang++", "-O1", "-std=c++17", "-fsanitize=undefined", "-fno-sanitize-recover=all", "-I", os.path.join(ROOT, "include"),
         "-c", str(drv), "-o", str(tmp_path / "driver.o")])
    run([HIPCC, "--offload-arch=gfx950", *san[:2], "-o", exe, str(tmp_path / "driver.o"), obj, "-Wl,-rpath,/opt/rocm/lib"])
    assert "0 wrong" in run([exe])
