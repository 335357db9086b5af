"""The sanitizer build of test_abi_sanitized for the checkpoint, transposed-product and adapter entry points: valid, empty,
extreme and invalid calls of each, on the CPU, against stub launchers."""
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
alignas(16) static unsigned char buf[4096];
static uint8_t* const P = buf;
static uint8_t* const F = buf + 4;  // 4-byte aligned only
static uint8_t* const H = buf + 2;  // less than that

struct Call {  // one that is valid, to be changed in one place at a time
  int64_t m = 4, k = 64, n = 5, l = 3, s = 2;
  int32_t g = 32, r = 8;
  int x = W4_BF16, sz = W4_F16, ab = W4_BF16, y = W4_F32;
  void *in = P, *packed = P, *scales = P, *zeros = P, *a = P, *b = P, *c = F, *o = F, *w = F, *low = P, *out = P, *ws = P;
  size_t bytes = sizeof(buf);
  int forward() const {
    return w4a16_lora_matmul(in, x, m, k, (uint8_t*)packed, scales, zeros, sz, n, g, a, b, ab, l, r, (float*)c, (int32_t*)o,
                             (int32_t*)w, s, (float*)low, out, y, ws, bytes, nullptr);
  }
  int back() const {
    return w4a16_lora_matmul_t(in, x, m, k, (uint8_t*)packed, scales, zeros, sz, n, g, a, b, ab, l, r, (float*)c, (int32_t*)o,
                               (int32_t*)w, s, (float*)low, out, y, ws, bytes, nullptr);
  }
  int plain() const {
    return w4a16_matmul_t(in, x, m, k, (uint8_t*)packed, scales, zeros, sz, n, g, out, y, ws, bytes, nullptr);
  }
  int grads() const {
    return lora_grads((int8_t*)in, (float*)c, m, k, packed, x, n, (float*)low, (float*)a, (int32_t*)o, (int32_t*)w, s, l, r,
                      (float*)b, (float*)out, ws, bytes, nullptr);
  }
};

int main() {
  const int64_t BIG = INT64_MAX, M32 = INT64_MAX - INT64_MAX % 32;
  // checkpoints
  for (int dt : {W4_F32, W4_BF16}) expect(quantize_checkpoint_int8(P, dt, 4, 160, (int8_t*)P, (float*)F, nullptr), W4_OK, "q ok");
  expect(quantize_checkpoint_int8(P, W4_F16, 4, 160, (int8_t*)P, (float*)F, nullptr), W4_EINVAL, "q f16");
  expect(quantize_checkpoint_int8(P, W4_F32, 1 << 24, 4096, (int8_t*)P, (float*)F, nullptr), W4_OK, "q 2^36");
  expect(quantize_checkpoint_int8(P, W4_F32, 1 << 24, 4128, (int8_t*)P, (float*)F, nullptr), W4_EINVAL, "q over 2^36");
  expect(quantize_checkpoint_int8(nullptr, W4_F32, 0, 32, nullptr, nullptr, nullptr), W4_OK, "q empty");
  expect(quantize_checkpoint_int8(P, W4_F32, 4, 32, (int8_t*)P, (float*)H, nullptr), W4_EINVAL, "q xs 2B");
  expect(quantize_checkpoint_int8(F, W4_F32, 4, 32, (int8_t*)P, (float*)F, nullptr), W4_EINVAL, "q x 4B");
  for (int64_t m : {(int64_t)-1, ((int64_t)1 << 24) + 1, BIG, INT64_MIN})
    expect(quantize_checkpoint_int8(P, W4_F32, m, 32, (int8_t*)P, (float*)F, nullptr), W4_EINVAL, "q m");
  for (int64_t k : {(int64_t)0, (int64_t)-32, (int64_t)16, (int64_t)100, ((int64_t)1 << 23) + 32, M32, INT64_MIN}) {
    expect(quantize_checkpoint_int8(P, W4_F32, 4, k, (int8_t*)P, (float*)F, nullptr), W4_EINVAL, "q k");
    expect(dequant_checkpoint_int8((int8_t*)P, (float*)F, 4, k, P, W4_F32, nullptr), W4_EINVAL, "dq k");
  }
  for (int dt : {W4_F32, W4_F16, W4_BF16}) expect(dequant_checkpoint_int8((int8_t*)P, (float*)F, 4, 160, P, dt, nullptr), W4_OK, "dq ok");
  for (int dt : {-1, 3, INT32_MAX, INT32_MIN})
    expect(dequant_checkpoint_int8((int8_t*)P, (float*)F, 4, 160, P, dt, nullptr), W4_EINVAL, "dq dtype");
  // products and gradients
  const Call ok;
  expect(ok.forward(), W4_OK, "forward ok");
  expect(ok.back(), W4_OK, "back ok");
  expect(ok.plain(), W4_OK, "plain ok");
  expect(ok.grads(), W4_OK, "grads ok");
  Call c;
  auto products = [&](int want, const char* what) {
    expect(c.forward(), want, what);
    expect(c.back(), want, what);
    expect(c.plain(), want, what);
    c = Call();
  };
  auto adapters = [&](int want, const char* what) {
    expect(c.forward(), want, what);
    expect(c.back(), want, what);
    c = Call();
  };
  auto all = [&](int want, const char* what) {
    expect(c.grads(), want, what);
    adapters(want, what);
  };
  for (int t : {W4_F32, W4_BF16}) { c.x = t; all(W4_OK, "x types"); c.ab = t; adapters(W4_OK, "ab types"); c.y = t; products(W4_OK, "y types"); }
  for (int t : {(int)W4_F16, -1, 3, INT32_MAX, INT32_MIN}) {
    c.x = t; products(W4_EINVAL, "x type");
    c.x = t; expect(c.grads(), W4_EINVAL, "dy type"); c = Call();
    c.ab = t; adapters(W4_EINVAL, "ab type");
    c.y = t; products(W4_EINVAL, "y type");
  }
  c.sz = W4_BF16; products(W4_EINVAL, "sz type");
  for (int32_t r : {0, -8, 4, 12, 264, INT32_MAX, INT32_MIN}) { c.r = r; all(W4_EINVAL, "rank"); }
  for (int32_t r : {8, 24, 256}) { c.r = r; all(W4_OK, "rank ok"); }
  for (int64_t v : {(int64_t)-1, (int64_t)65537, BIG, INT64_MIN}) { c.l = v; all(W4_EINVAL, "adapters"); }
  for (int64_t v : {(int64_t)-1, ((int64_t)1 << 20) + 1, BIG, INT64_MIN}) { c.s = v; all(W4_EINVAL, "segments"); }
  c.l = 65536; c.s = 1 << 20; all(W4_OK, "most adapters and segments");
  c.l = 65536; c.r = 256; c.k = 4096; all(W4_OK, "l r k = 2^36");
  c.l = 65536; c.r = 256; c.k = 4128; all(W4_EINVAL, "l r k over");
  c.l = 65536; c.r = 256; c.n = 4097; all(W4_EINVAL, "l r n over");
  for (int64_t m : {(int64_t)-1, ((int64_t)1 << 24) + 1, BIG, INT64_MIN}) {
    c.m = m; all(W4_EINVAL, "m");
    c.m = m; products(W4_EINVAL, "m");
  }
  for (int64_t k : {(int64_t)0, (int64_t)-32, (int64_t)48, M32, INT64_MIN}) {
    c.k = k; all(W4_EINVAL, "k");
    c.k = k; products(W4_EINVAL, "k");
  }
  for (int64_t n : {(int64_t)-1, BIG, INT64_MIN}) { c.n = n; all(W4_EINVAL, "n"); c.n = n; products(W4_EINVAL, "n"); }
  for (int32_t g : {0, -32, 48, INT32_MAX, INT32_MIN}) { c.g = g; products(W4_EINVAL, "g"); }
  // empty calls
  Call none;
  none.in = none.packed = none.scales = none.zeros = none.a = none.b = none.c = none.o = none.w = none.low = none.out = none.ws = nullptr;
  none.bytes = 0;
  c = none; c.m = 0; products(W4_OK, "m = 0");
  c = none; c.n = 0; expect(c.forward(), W4_OK, "n = 0 forward");
  expect(c.back(), W4_EINVAL, "n = 0 back"); expect(c.plain(), W4_EINVAL, "n = 0 plain");
  c = none; c.l = 0; expect(c.grads(), W4_OK, "no adapters");
  c = Call(); c.l = 0; c.a = c.b = c.c = c.o = c.w = c.low = nullptr; adapters(W4_OK, "no adapters");
  c.s = 0; c.a = c.b = c.c = c.o = c.w = c.low = nullptr; adapters(W4_OK, "no segments");
  c.s = 0; c.in = c.c = c.packed = c.low = c.a = c.o = c.w = nullptr; expect(c.grads(), W4_OK, "grads without segments");
  // pointers, one at a time
  void* Call::*const full[] = {&Call::in, &Call::packed, &Call::scales, &Call::zeros, &Call::out};
  for (auto p : full)
    for (void* v : {(void*)nullptr, (void*)F}) { c = Call(); c.*p = v; products(W4_EINVAL, "pointer"); }
  void* Call::*const low[] = {&Call::a, &Call::b, &Call::low};
  for (auto p : low)
    for (void* v : {(void*)nullptr, (void*)F}) { c = Call(); c.*p = v; all(W4_EINVAL, "adapter pointer"); }
  void* Call::*const four[] = {&Call::c, &Call::o, &Call::w};
  for (auto p : four)
    for (void* v : {(void*)nullptr, (void*)H}) { c = Call(); c.*p = v; all(W4_EINVAL, "4-byte pointer"); }
  // sizes of workspaces: whatever the arguments, an answer
  for (int64_t m : {(int64_t)-1, (int64_t)0, (int64_t)7, (int64_t)1 << 24, BIG, INT64_MIN})
    for (int64_t k : {(int64_t)0, (int64_t)64, (int64_t)1 << 23, M32, INT64_MIN})
      for (int64_t n : {(int64_t)0, (int64_t)5, BIG, INT64_MIN}) {
        (void)w4a16_lora_matmul_workspace_size(m, k, n, 32, W4_BF16, W4_F16, W4_F32);
        (void)w4a16_matmul_t_workspace_size(m, k, n, 0, 9, -1, W4_BF16);
        (void)lora_grads_workspace_size(m, k, n, W4_BF16, 65536, 256);
        (void)lora_grads_workspace_size(m, k, n, 7, INT64_MIN, INT32_MIN);
      }
  std::printf("driver done, %d failure(s)\n", fails);
  return fails != 0;
}
'''


def test_adapter_entry_points_under_sanitizers(tmp_path):
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
    assert r.returncode == 0 and "driver done, 0 failure(s)" in r.stdout, r.stdout[-3000:] + r.stderr[-3000:]
