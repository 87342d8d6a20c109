"""How the parts of a row's largest logit and sum are joined in the verification of drafts (csrc/peak.h).

Lanes, warps and blocks join the same parts in butterflies, each with its own part first, and then walk a tree by what
they got: the results have to be the same bits everywhere. The source that the kernel includes is compiled here for the
host, with a compiler that may fuse products and sums as nvcc may.
"""
import ctypes
import os
import platform
import subprocess

import numpy as np
import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "moe_expert_layer_top_gb300", "csrc")

SHIM = r"""
#include <cmath>
#define __device__
#define __forceinline__ inline
// rounded each by itself, as CUDA's of these names are
static __attribute__((noinline)) float __fmul_rn(float a, float b) { return a * b; }
static __attribute__((noinline)) float __fadd_rn(float a, float b) { return a + b; }
#include "peak.h"

struct Plain : moe::Peak {  // the same left to the compiler
  template <class F>
  inline void join(const Plain &o, float c, F exp2) {
    const float t = fmaxf(top, o.top), ref = t == -INFINITY ? 0.0f : t;
    sum = sum * exp2((top - ref) * c) + o.sum * exp2((o.top - ref) * c);
    if (o.top > top || (o.top == top && o.token < token)) token = o.token;
    top = t;
  }
};

template <class P>
static void butterfly(P *k, int n, float c) {
  P next[64];
  for (int d = n / 2; d; d /= 2) {
    for (int i = 0; i < n; ++i) {
      next[i] = k[i];
      next[i].join(k[i ^ d], c, [](float x) { return std::exp2(x); });
    }
    for (int i = 0; i < n; ++i) k[i] = next[i];
  }
}

extern "C" void join(int plain, int n, float *top, float *sum, int *token, float c) {
  moe::Peak k[64];
  Plain p[64];
  for (int i = 0; i < n; ++i) k[i] = {top[i], sum[i], token[i]}, static_cast<moe::Peak &>(p[i]) = k[i];
  if (plain)
    butterfly(p, n, c);
  else
    butterfly(k, n, c);
  for (int i = 0; i < n; ++i) {
    const moe::Peak &r = plain ? p[i] : k[i];
    top[i] = r.top, sum[i] = r.sum, token[i] = r.token;
  }
}
"""


def fuses():
    """Flags with which the host's compiler fuses; None where the machine cannot."""
    if platform.machine() == "x86_64":
        with open("/proc/cpuinfo") as f:
            return ["-mfma"] if " fma " in f.read() else None
    return [] if platform.machine() == "aarch64" else None


@pytest.fixture(scope="module")
def join(tmp_path_factory):
    flags = fuses()
    if flags is None:
        pytest.skip("no fused multiply-add here")
    at = tmp_path_factory.mktemp("join")
    (at / "join.cpp").write_text(SHIM)
    subprocess.run([os.environ.get("CXX") or "g++", "-O2", "-std=c++17", "-ffp-contract=fast", *flags, "-fPIC", "-shared", "-I",
                    CSRC, str(at / "join.cpp"), "-o", str(at / "join.so")], check=True)
    lib = ctypes.CDLL(str(at / "join.so"))

    def call(plain, top, sum, token, c):
        arrays = [np.array(top, np.float32), np.array(sum, np.float32), np.array(token, np.int32)]
        lib.join(int(plain), len(top), *(a.ctypes.data_as(ctypes.c_void_p) for a in arrays), ctypes.c_float(c))
        return arrays

    return call


def parts(seed):
    rng = np.random.default_rng(seed)
    n = int(rng.choice([8, 32]))
    top = rng.normal(0, rng.choice([0.1, 1.0, 10.0]), n).astype(np.float32)
    if seed % 5 == 0:  # parts without a logit, and equal ones
        top[rng.integers(0, n, 3)] = -np.inf
        top[rng.integers(0, n, 3)] = top.max()
    sum = np.where(np.isneginf(top), 0.0, rng.uniform(1.0, 300.0, n)).astype(np.float32)
    return top, sum, rng.permutation(n).astype(np.int32), np.float32(1.4426950408889634 / rng.choice([0.7, 1.0, 1.3]))


@pytest.mark.parametrize("seed", range(200))
def test_every_lane_gets_the_same(join, seed):
    top, sum, token, c = parts(seed)
    t, s, k = join(False, top, sum, token, c)
    assert len(np.unique(t)) == 1 and len(np.unique(s.view(np.uint32))) == 1 and len(np.unique(k)) == 1
    assert t[0] == top.max() and k[0] == token[top == top.max()].min()
    want = (sum.astype(np.float64) * np.exp2((top.astype(np.float64) - top.max()) * float(c))).sum()
    # a factor's argument has two roundings, its value one; then a product and a sum for each of log2(n) joins
    wide = np.where(np.isneginf(top), 0.0, top.max() - top).max() * float(c)
    assert abs(s[0] - want) <= want * 2.0 ** -24 * 5 * (2 * wide + 4)


def test_the_plain_form_would_not_do(join):
    """What the above is for: left to the compiler the lanes get different sums."""
    different = 0
    for seed in range(200):
        top, sum, token, c = parts(seed)
        different += len(np.unique(join(True, top, sum, token, c)[1].view(np.uint32))) > 1
    assert different > 50


def test_parts_without_a_logit(join):
    none = np.full(32, -np.inf, np.float32)
    t, s, k = join(False, none, np.zeros(32), np.full(32, 2 ** 31 - 1), 1.0)
    assert np.isneginf(t).all() and (s == 0).all() and (k == 2 ** 31 - 1).all()
