"""Pins of the oracle's rotation, cache rows and attention (CPU), and the
cache's address arithmetic compiled for the host."""

import os
import shutil
import subprocess

import numpy as np
import pytest

import oracle

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def test_rope_hand_worked():
    """A quarter turn maps (a, b) to (-b, a); far positions keep the angle."""
    x = np.arange(1, 9, dtype=np.float64).reshape(1, 1, 8)
    f = np.float32(0.5)
    y = oracle.rope_ref(x, [2], [f, 0.0], interleaved=True)
    c, s = np.cos(1.0), np.sin(1.0)
    assert np.allclose(y[0, 0], [c - 2 * s, s + 2 * c, 3, 4, 5, 6, 7, 8], atol=1e-15)
    y = oracle.rope_ref(x, [2], [f, 0.0])
    assert np.allclose(y[0, 0], [c - 3 * s, 2, s + 3 * c, 4, 5, 6, 7, 8], atol=1e-15)
    # 2^30 * 0.1f is an exact rational: its angle by integer arithmetic modulo 2 pi
    import fractions
    th = fractions.Fraction(2**30) * fractions.Fraction(float(np.float32(0.1)))
    two_pi = fractions.Fraction("6.28318530717958647692528676655900576839433879875021")
    th = float(th - (th // two_pi) * two_pi)
    y = oracle.rope_ref(np.array([[[1.0, 0.0]]]), [2**30], [np.float32(0.1)], interleaved=True)
    assert np.allclose(y[0, 0], [np.cos(th), np.sin(th)], atol=1e-9)
    z = oracle.rope_ref(x, [5], [f, f], norm=True, eps=0.0)
    assert np.isclose(np.sum(z * z), 8.0)  # a rotation keeps the norm


@pytest.mark.parametrize("fmt", oracle.KV_FMTS)
@pytest.mark.parametrize("D", [64, 128, 256])
def test_cache_rows_round_trip(fmt, D):
    rng = np.random.default_rng(D)
    x = rng.standard_normal((5, 3, D)).astype(np.float32)
    codes, scales = oracle.kv_encode(fmt, x)
    assert codes.shape[-1] + scales.shape[-1] == {"bf16": 2 * D, "q8_0": D * 17 // 16, "q4_0": D * 9 // 16}[fmt]
    y = oracle.kv_decode(fmt, codes, scales)
    step = {"bf16": 2.0**-8 * np.abs(x), "q8_0": 0, "q4_0": 0}[fmt]
    if fmt != "bf16":
        b = np.abs(x).reshape(5, 3, -1, 32).max(-1)
        step = np.repeat(b * (0.51 / 127 if fmt == "q8_0" else 1.01 / 8), 32, -1)
    assert np.all(np.abs(y - x) <= step + 1e-3 * np.abs(x) * (fmt != "bf16"))
    # decoded values are fixed points
    again = oracle.kv_decode(fmt, *oracle.kv_encode(fmt, y.astype(np.float32)))
    if fmt == "bf16":
        assert np.array_equal(again, y)


def test_row_places_are_a_permutation():
    for D in (64, 128, 256):
        p = oracle.row_places(D)
        assert sorted(p) == list(range(D))
        assert p[0] == 0 and p[1] == 1 and p[32] == 2 and p[2] == D // 16


def test_extreme_scale_stays_finite():
    x = np.full((1, 64), 3e38, np.float32)
    for fmt in ("q8_0", "q4_0"):
        assert np.all(np.isfinite(oracle.kv_decode(fmt, *oracle.kv_encode(fmt, x))))


def test_attention_hand_worked():
    q = np.zeros((2, 1, 64))
    k = np.zeros((3, 1, 64))
    v = np.stack([np.full((1, 64), t) for t in (1.0, 2.0, 6.0)])
    o, a, e = oracle.tree_attn_ref(q, k, v, np.array([[1, 1, 1], [0, 0, 0]], bool), 1.0)
    assert np.allclose(o[0], 3.0) and np.all(o[1] == 0)
    k[2], q[0] = 1.0, 1.0
    v[1] = np.nan  # not seen
    o, _, _ = oracle.tree_attn_ref(q, k, v, np.array([[1, 0, 1], [0, 0, 0]], bool), 0.01)
    w = np.exp(0.64)
    assert np.allclose(o[0], (1 + 6 * w) / (1 + w))


_LAYOUT_MAIN = r"""
#include "kv_layout.h"
#include <cstdio>
#include <cstdlib>
#include <vector>
using namespace skg;
#define CHECK(c) do { if (!(c)) { std::printf("line %d: %s\n", __LINE__, #c); std::exit(1); } } while (0)
int main() {
  // every slot of small caches: offsets in range, codes and scales of all slots apart
  for (int kind = 0; kind < 3; ++kind)
    for (int D : {64, 128, 256})
      for (uint32_t shift : {4u, 6u})
        for (uint32_t heads : {1u, 3u}) {
          const int64_t pages = 3;
          KvView c{nullptr, nullptr, pages, heads, shift, uint32_t((kv_row_bytes(kind, D) + kv_scale_bytes(kind, D)) << shift)};
          const uint64_t bytes = uint64_t(pages) * heads * c.chunk;
          std::vector<int> used(bytes, 0);
          CHECK(c.chunk % 16 == 0);
          for (int64_t s = -70; s < (pages << shift) + 70; ++s) {
            if (!kv_slot_in(c, s)) { CHECK(s < 0 || s >= (pages << shift)); continue; }
            for (uint32_t h = 0; h < heads; ++h) {
              const uint64_t at = kv_chunk_at(c, s >> shift, h);
              const uint32_t t = uint32_t(s & ((1 << shift) - 1));
              for (uint32_t i = 0; i < kv_row_bytes(kind, D); ++i) CHECK(at + kv_codes_at(kind, D, t) + i < bytes && !used[at + kv_codes_at(kind, D, t) + i]++);
              for (uint32_t i = 0; i < kv_scale_bytes(kind, D); ++i) CHECK(at + kv_scales_at(kind, D, shift, t) + i < bytes && !used[at + kv_scales_at(kind, D, shift, t) + i]++);
            }
          }
          for (int u : used) CHECK(u == 1);
        }
  KvView big{nullptr, nullptr, 2147483647, 65535, 20, 512u << 20};
  CHECK(kv_slot_in(big, (int64_t(2147483647) << 20) - 1) && !kv_slot_in(big, int64_t(2147483647) << 20));
  CHECK(!kv_slot_in(big, INT64_MIN) && !kv_slot_in(big, INT64_MAX));
  CHECK(kv_page_in(big, 0) && kv_page_in(big, 2147483646) && !kv_page_in(big, 2147483647) && !kv_page_in(big, -1) && !kv_page_in(big, INT32_MIN));
  CHECK(kv_chunk_at(big, 100000, 7) == (uint64_t(100000) * 65535 + 7) * (512u << 20));
  // spans: whatever the device arrays hold, tokens lie in [0, T) and keys in [0, max_kv]
  const int32_t some[] = {INT32_MIN, -5, -1, 0, 1, 3, 7, 8, 9, 63, 64, 65, 100, 2147483600, INT32_MAX};
  for (int64_t T : {1, 8, 70})
    for (int md : {1, 8, 64})
      for (int64_t mk : {int64_t(16), int64_t(64), int64_t(2147483583)})
        for (int32_t ctx : some)
          for (int32_t a : some)
            for (int32_t b : some) {
              const KvSpan s = kv_span(ctx, a, b, T, md, mk);
              CHECK(s.n >= 0 && s.n <= md && s.t0 >= 0 && int64_t(s.t0) + s.n <= T);
              CHECK(s.ctx >= 0 && s.ctx <= s.keys && s.keys <= mk && s.keys <= int64_t(s.ctx) + s.n);
              if (ctx >= 0 && a >= 0 && b >= a && b <= T && b - a <= md && int64_t(ctx) + b - a <= mk)
                CHECK(s.t0 == a && s.n == b - a && s.ctx == ctx && s.keys == ctx + b - a);
            }
  std::puts("ok");
}
"""


def test_cache_addresses_on_the_host(tmp_path):
    """Slots and pages outside a cache, lengths and token ranges outside their
    arrays: the kernels' own bounds arithmetic, compiled for the CPU."""
    cxx = shutil.which("g++")
    if cxx is None:
        pytest.skip("no host compiler")
    src, exe = tmp_path / "t.cpp", tmp_path / "t"
    src.write_text(_LAYOUT_MAIN)
    subprocess.run([cxx, "-std=c++17", "-O1", "-fsanitize=undefined", "-fno-sanitize-recover", "-I",
                    os.path.join(ROOT, "skinny_gemm_decode_amd", "csrc"), str(src), "-o", str(exe)], check=True)
    r = subprocess.run([str(exe)], capture_output=True, text=True, timeout=60)
    assert r.returncode == 0 and r.stdout.strip() == "ok", r.stdout + r.stderr


_SPLIT_MAIN = r"""
#include <cstdio>
#include <cstdlib>
#include <random>
#include <vector>
#include "kv_layout.h"
using namespace skg;
#define CHECK(x) do { if (!(x)) { std::printf("line %d: %s\n", __LINE__, #x); return 1; } } while (0)
int main() {
  std::mt19937 rng(5);
  const int64_t bounds[] = {0, 1, 32, 100, 5000, 131072, int64_t(1) << 26, int64_t(INT32_MAX) - 64};
  for (int trial = 0; trial < 20000; ++trial) {
    const int64_t max_kv = bounds[rng() % 8];
    const int n_seqs = 1 + rng() % (trial & 1 ? 256 : 4), want = 1 + rng() % (trial & 2 ? 1024 : 3);
    const bool weigh = trial & 4;
    const int shift = kv_cost_shift(max_kv, n_seqs);
    CHECK(shift >= 0 && shift < 16);
    std::vector<int> steps(n_seqs), each(n_seqs);
    int64_t total = 0;
    const int kind = rng() % 3;  // all as long as they may be, any, a few long ones
    for (int b = 0; b < n_seqs; ++b) {
      const int64_t keys = kind == 0 ? max_kv : kind == 1 || rng() % 8 == 0 ? int64_t(rng()) % (max_kv + 1) : rng() % 5;
      steps[b] = kv_steps(int32_t(keys < max_kv ? keys : max_kv));
      each[b] = !weigh ? 1 : rng() % 2 ? kMaxWeight : 3;
      total += kv_cost(steps[b], each[b], shift);
    }
    CHECK(total <= INT32_MAX);
    const int cost = int(total) / want + (int(total) % want != 0);
    int64_t splits = 0;
    const int64_t most = (((max_kv + kStep - 1) / kStep) + kMinSteps - 1) / kMinSteps;
    for (int b = 0; b < n_seqs; ++b) {
      const int per = kv_split_steps(cost, each[b], shift), n = kv_splits(steps[b], per);
      CHECK(per >= kMinSteps && n >= 1 && n <= (most < 1 ? 1 : most));
      CHECK(int64_t(per) * n >= steps[b] && int64_t(per) * (n - 1) < (steps[b] ? steps[b] : 1));
      CHECK(int64_t(per) * n <= INT32_MAX);  // no overflow in a split's end
      splits += n;
    }
    CHECK(splits <= int64_t(want) + n_seqs);
  }
  std::puts("ok");
}
"""


def test_splits_fit_their_workspace_on_the_host(tmp_path):
    """At most want + n_seqs splits, whatever the lengths: the arithmetic of the
    kernels, compiled for the CPU."""
    cxx = shutil.which("g++")
    if cxx is None:
        pytest.skip("no host compiler")
    src, exe = tmp_path / "s.cpp", tmp_path / "s"
    src.write_text(_SPLIT_MAIN)
    subprocess.run([cxx, "-std=c++17", "-O1", "-fsanitize=undefined", "-fno-sanitize-recover", "-I",
                    os.path.join(ROOT, "skinny_gemm_decode_amd", "csrc"), str(src), "-o", str(exe)], check=True)
    r = subprocess.run([str(exe)], capture_output=True, text=True, timeout=60)
    assert r.returncode == 0 and r.stdout.strip() == "ok", r.stdout + r.stderr
