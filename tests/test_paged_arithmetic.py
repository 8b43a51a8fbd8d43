"""The arithmetic in two fp32 numbers that decides a 4-bit cache's codes,
compiled for the host and compared with long double."""
import ctypes
import os
import subprocess

import pytest

from cross_model_attention_gb300 import build as build_mod

SOURCE = r"""
#include "mf_ff.cuh"
#include <cmath>
#include <cstdint>
using namespace mf;
static long double of(ff x) { return static_cast<long double>(x.h) + x.l; }
// A generator of its own: 64 bits at a time (xorshift64*).
static uint64_t next(uint64_t& s) {
  s ^= s >> 12, s ^= s << 25, s ^= s >> 27;
  return s * 2685821657736338717ull;
}
static double worse(double a, long double x) { return std::fabs(static_cast<double>(x)) > a ? std::fabs(static_cast<double>(x)) : a; }
static double off(uint64_t turn) {
  // the angle in long double, to the nearest quarter turn exactly
  const unsigned quarter = static_cast<unsigned>((turn + (1ull << 61)) >> 62) & 3u;
  const int64_t r = static_cast<int64_t>(turn - (static_cast<uint64_t>(quarter) << 62));
  const long double a = ldexpl(static_cast<long double>(r), -64) * 6.283185307179586476925286766559L;
  const long double s = sinl(a), c = cosl(a);
  const long double sn = quarter == 0 ? s : quarter == 1 ? c : quarter == 2 ? -s : -c;
  const long double cn = quarter == 0 ? c : quarter == 1 ? -s : quarter == 2 ? -c : s;
  ff fs, fc;
  ff_sincos(turn, &fs, &fc);
  return worse(worse(0, of(fs) - sn), of(fc) - cn);
}
extern "C" double sincos_off(int random) {
  double w = 0;
  for (uint64_t j = 0; j < 128; ++j)        // 64ths of a turn, quarters and eighths, and the middles between 64ths
    for (int64_t e = -5; e <= 5; ++e)
      for (int k = 0; k < 60; k += 7) w = worse(w, off((j << 57) + static_cast<uint64_t>(e * (1ll << k))));
  for (int k = 0; k < 64; ++k) w = worse(worse(w, off(1ull << k)), off(0ull - (1ull << k)));
  uint64_t s = 88172645463325252ull;
  for (int i = 0; i < random; ++i) w = worse(w, off(next(s)));
  return w;
}
static ff some(uint64_t& s) {  // 2^-20 .. 2^20 in two parts
  const double x = ldexp(static_cast<double>(static_cast<int64_t>(next(s))), static_cast<int>(next(s) % 41) - 83);
  const float h = static_cast<float>(x);
  return {h, static_cast<float>(x - h)};
}
extern "C" double product_off(int random) {  // relative
  double w = 0;
  uint64_t s = 1234567;
  for (int i = 0; i < random; ++i) {
    const ff a = some(s), b = some(s);
    w = worse(w, (of(ff_mul(a, b)) - of(a) * of(b)) / (of(a) * of(b)));
    w = worse(w, (of(ff_mul(a, b.h)) - of(a) * b.h) / (of(a) * b.h));
  }
  return w;
}
extern "C" double sum_off(int random) {  // of |a| + |b|
  double w = 0;
  uint64_t s = 7654321;
  for (int i = 0; i < random; ++i) {
    const ff a = some(s);
    ff b = some(s);
    if (i % 3 == 0) b = ff_neg({a.h * (1.f + (i % 5) * 0x1p-23f), a.l * 0.75f});
    w = worse(w, (of(ff_add(a, b)) - of(a) - of(b)) / (fabsl(of(a)) + fabsl(of(b))));
    const ff e = ff_sum(a.h, b.h);
    if (of(e) != static_cast<long double>(a.h) + b.h) return 1;  // (error-free, 2^41 between them at most)
  }
  return w;
}
"""


@pytest.fixture(scope="module")
def lib(tmp_path_factory):
    d = tmp_path_factory.mktemp("ff")
    src, out = str(d / "ff.cpp"), str(d / "libff.so")
    with open(src, "w") as f:
        f.write(SOURCE)
    # (with sums and products fused where the machine can: sums and products stay as they are written all the same)
    r = subprocess.run(["g++", "-std=c++17", "-O3", "-ffp-contract=fast", "-shared", "-fPIC", "-I", build_mod.CSRC, src, "-o", out],
                       capture_output=True, text=True)
    assert r.returncode == 0, r.stderr
    lib = ctypes.CDLL(out)
    for name in ("sincos_off", "product_off", "sum_off"):
        getattr(lib, name).restype = ctypes.c_double
    return lib


def test_sine_and_cosine_of_a_turn(lib):
    # of the rest d <= pi / 64: d^4 / 24 <= 2^-21.98 comes from fp32, d^2's high part, a square, a
    # product and a sum's rest, 5 roundings of 2^-24 at most: 2^-43.6; the next term d^8 / 40320 is
    # below 2^-49, the table and the products and sums of two parts are good to 2^-46 together
    assert lib.sincos_off(300000) <= 2.0 ** -43


def test_products_of_two_parts(lib):
    # what is left out (low times low) is 2^-48 of the product; three roundings of a rest of 2^-23 of it at most
    assert lib.product_off(300000) <= 3 * 2.0 ** -47 + 2.0 ** -48 + 2.0 ** -47


def test_sums_of_two_parts(lib):
    # two roundings of the low parts' sums, each at most 2^-23 (|a| + |b|), and the last one's
    assert lib.sum_off(300000) <= 3 * 2.0 ** -47
