"""The sanitizer build of test_abi_sanitized for the MXFP4 and by-expert entry
points: valid, empty, extreme and invalid calls of each, on the CPU, against
stub launchers.  The 64-bit products of experts, rows and columns are what it is for."""
import os
import subprocess


from tests import test_abi_sanitized as base

pytestmark = base.pytestmark

DRIVER = r'''
#include <cstdint>
#include <cstdio>
#include "w4.h"

static int fails = 0;
static void expect(int got, int want, const char* what) {
  if (got != want) {
    std::printf("%s: status %d, expected %d (%s)\n", what, got, want, w4_last_error());
    ++fails;
  }
}

int main() {
  alignas(16) static unsigned char buf[4096];
  uint8_t* P = buf;
  uint8_t* F = buf + 4;  // 4-byte aligned only
  uint8_t* B = buf + 2;  // less than that
  const int32_t* O = (const int32_t*)buf;
  const int64_t BIG = INT64_MAX, M32 = INT64_MAX - INT64_MAX % 32;
  // quantize, dequantize
  expect(quantize_mxfp4(P, W4_BF16, 4, 256, P, F, nullptr), W4_OK, "q ok, scales 4B");
  expect(quantize_mxfp4(P, W4_F32, 1LL << 31, 32, P, P, nullptr), W4_OK, "q 2^36 elements");
  expect(quantize_mxfp4(P, W4_F32, (1LL << 31) + 1, 32, P, P, nullptr), W4_EINVAL, "q over 2^36");
  expect(quantize_mxfp4(P, W4_BF16, BIG, 32, P, P, nullptr), W4_EINVAL, "q n huge");
  expect(quantize_mxfp4(P, W4_BF16, 4, M32, P, P, nullptr), W4_EINVAL, "q k huge");
  expect(quantize_mxfp4(P, W4_BF16, INT64_MIN, 32, P, P, nullptr), W4_EINVAL, "q n least");
  expect(quantize_mxfp4(P, W4_BF16, 4, INT64_MIN, P, P, nullptr), W4_EINVAL, "q k least");
  expect(quantize_mxfp4(F, W4_BF16, 4, 32, P, P, nullptr), W4_EINVAL, "q w 4B");
  expect(quantize_mxfp4(P, W4_BF16, 4, 32, P, B, nullptr), W4_EINVAL, "q scales 2B");
  expect(quantize_mxfp4(nullptr, W4_BF16, 0, 32, nullptr, nullptr, nullptr), W4_OK, "q empty");
  for (int dt : {-1, 3, INT32_MAX, INT32_MIN}) expect(quantize_mxfp4(P, dt, 4, 32, P, P, nullptr), W4_EINVAL, "q dtype");
  for (int dt : {W4_F32, W4_F16, W4_BF16}) expect(dequant_mxfp4(P, F, 4, 256, P, dt, nullptr), W4_OK, "dq ok");
  expect(dequant_mxfp4(P, P, BIG, M32, P, W4_F32, nullptr), W4_EINVAL, "dq huge");
  expect(dequant_mxfp4(P, P, 4, 256, F, W4_F32, nullptr), W4_EINVAL, "dq out 4B");
  // the dense product
  for (int64_t m : {1, 16, 33, 129, 2048}) expect(mxfp4_matmul(P, F, m, 4096, P, F, 11008, P, W4_BF16, nullptr), W4_OK, "mm ok");
  expect(mxfp4_matmul(P, P, 0x7fffffffLL, 32, P, P, 1, P, W4_F32, nullptr), W4_OK, "mm m most");
  expect(mxfp4_matmul(P, P, 0x80000000LL, 32, P, P, 1, P, W4_F32, nullptr), W4_EINVAL, "mm m over");
  expect(mxfp4_matmul(P, P, BIG, M32, P, P, BIG, P, W4_F32, nullptr), W4_EINVAL, "mm huge");
  expect(mxfp4_matmul(P, P, 5, 1 << 23, P, P, 8192, P, W4_F32, nullptr), W4_OK, "mm k most");
  expect(mxfp4_matmul(P, P, 5, (1 << 23) + 32, P, P, 1, P, W4_F32, nullptr), W4_EINVAL, "mm k over");
  expect(mxfp4_matmul(P, P, 0, 32, nullptr, nullptr, 5, nullptr, W4_F32, nullptr), W4_OK, "mm empty");
  expect(mxfp4_matmul(P, P, 5, 32, P, P, 5, nullptr, W4_F32, nullptr), W4_EINVAL, "mm y null");
  // by expert: rows, experts and their products at and past the limits
  struct { int64_t t, k, e, n; int want; const char* what; } c[] = {
      {4, 64, 3, 5, W4_OK, "ok"},
      {1 << 24, 64, 65536, 5, W4_OK, "t and e most"},
      {(1 << 24) + 1, 64, 3, 5, W4_EINVAL, "t over"},
      {4, 64, 65537, 5, W4_EINVAL, "e over"},
      {4, 64, BIG, 5, W4_EINVAL, "e huge"},
      {4, 64, INT64_MIN, 5, W4_EINVAL, "e least"},
      {-1, 64, 3, 5, W4_EINVAL, "t < 0"},
      {BIG, 64, 3, 5, W4_EINVAL, "t huge"},
      {4, 64, 65536, 1 << 14, W4_OK, "e n k = 2^36"},
      {4, 64, 65536, (1 << 14) + 1, W4_EINVAL, "e n k over"},
      {4, 64, 3, BIG, W4_EINVAL, "n huge"},
      {4, M32, 3, 5, W4_EINVAL, "k huge"},
      {1 << 24, 1 << 12, 1, 5, W4_OK, "t k = 2^36"},
      {1 << 24, 1 << 13, 1, 5, W4_EINVAL, "t k over"},
      {1 << 24, 64, 1, 1 << 12, W4_OK, "t n = 2^36"},
      {1 << 24, 64, 1, 1 << 13, W4_EINVAL, "t n over"},
      {0, 64, 3, 5, W4_OK, "t = 0"},
      {4, 64, 0, 5, W4_OK, "e = 0"},
      {4, 64, 3, 0, W4_OK, "n = 0"},
  };
  for (const auto& a : c) {
    expect(mxfp4_grouped_matmul(P, F, a.t, a.k, (const int32_t*)F, a.e, P, F, a.n, P, W4_F32, nullptr), a.want, a.what);
    for (int xd : {W4_F32, W4_BF16})
      for (int g : {32, 64})
        expect(w4a16_grouped_matmul(P, xd, a.t, a.k, (const int32_t*)F, a.e, P, P, P, W4_F16, a.n, g, P, W4_BF16, nullptr),
               a.want, a.what);
  }
  expect(mxfp4_grouped_matmul(P, P, 4, 64, (const int32_t*)B, 3, P, P, 5, P, W4_F32, nullptr), W4_EINVAL, "offsets 2B");
  expect(mxfp4_grouped_matmul(P, P, 4, 64, nullptr, 3, P, P, 5, P, W4_F32, nullptr), W4_EINVAL, "offsets null");
  for (int g : {0, -32, 48, INT32_MIN, INT32_MAX})
    expect(w4a16_grouped_matmul(P, W4_BF16, 4, 64, O, 3, P, P, P, W4_F16, 5, g, P, W4_BF16, nullptr), W4_EINVAL, "g");
  expect(w4a16_grouped_matmul(P, W4_F16, 4, 64, O, 3, P, P, P, W4_F16, 5, 32, P, W4_BF16, nullptr), W4_EINVAL, "x f16");
  expect(w4a16_grouped_matmul(P, W4_F32, 4, 64, O, 3, P, P, P, W4_BF16, 5, 32, P, W4_BF16, nullptr), W4_EINVAL, "sz bf16");
  std::printf("driver done, %d failure(s)\n", fails);
  return fails != 0;
}
'''


def test_new_entry_points_under_sanitizers(tmp_path):
    (tmp_path / "stubs.cpp").write_text(base._stubs())
    (tmp_path / "driver.cpp").write_text(DRIVER)
    exe = tmp_path / "abi_san"
    flags = ["-std=c++17", "-g", "-O1", "-D__HIP_PLATFORM_AMD__", f"-I{base.ROCM}/include", f"-I{base.CSRC}",
             f"-I{os.path.join(base.ROOT, 'include')}", "-fsanitize=address,undefined", "-fno-sanitize-recover=all",
             "-fno-omit-frame-pointer"]
    cmd = ["g++", *flags, os.path.join(base.CSRC, "api.cpp"), str(tmp_path / "stubs.cpp"), str(tmp_path / "driver.cpp"),
           f"-L{base.ROCM}/lib", "-lamdhip64", "-o", str(exe)]
    r = subprocess.run(cmd, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stderr[-3000:]
    env = dict(os.environ, LD_LIBRARY_PATH=f"{base.ROCM}/lib:" + os.environ.get("LD_LIBRARY_PATH", ""),
               ASAN_OPTIONS="detect_leaks=0", UBSAN_OPTIONS="print_stacktrace=1")
    r = subprocess.run([str(exe)], capture_output=True, text=True, timeout=120, env=env)
    assert r.returncode == 0, (r.stdout + r.stderr)[-3000:]
    assert "driver done, 0 failure(s)" in r.stdout
