"""Pins of the windowed-attention oracle (no GPU), and of the units that a decode visits."""
import os
import subprocess

import numpy as np
import pytest

import oracle

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "paged_attention_kv_decode_gb300", "csrc")


def pages(rng, lens, G, D, bs):
    table = np.full((len(lens), max(1, max(-(-n // bs) for n in lens))), -1)
    order = rng.permutation(sum(-(-n // bs) for n in lens) + 2)
    at = 0
    for s, n in enumerate(lens):
        m = -(-n // bs)
        table[s, :m] = order[at:at + m]
        at += m
    return rng.standard_normal((len(order), bs, G, D)), rng.standard_normal((len(order), bs, G, D)), table


def test_tokens_by_hand():
    assert oracle.window_tokens(9, 3, 2).tolist() == [0, 1, 7, 8, 9]
    assert oracle.window_tokens(3, 3, 2).tolist() == [0, 1, 2, 3]
    assert oracle.window_tokens(5, 1, 0).tolist() == [5]
    assert oracle.window_tokens(2, 100, 100).tolist() == [0, 1, 2]


def test_wide_windows_are_plain_attention():
    rng = np.random.default_rng(0)
    lens, cu = [7, 1, 20], [0, 3, 4, 13]
    k, v, table = pages(rng, lens, 2, 8, 4)
    q = rng.standard_normal((13, 4, 8))
    want = oracle.paged_prefill(q, cu, k, v, table, lens, 0.3)
    for window, sinks in ((20, 0), (1000, 5), (1, 20)):
        got = oracle.paged_window(q, cu, k, v, table, lens, 0.3, window, sinks)
        assert np.allclose(got[0], want[0], atol=1e-13) and np.allclose(got[1], want[1], atol=1e-13)


def test_a_row_is_plain_attention_over_its_tokens():
    rng = np.random.default_rng(1)
    lens = [30]
    k, v, table = pages(rng, lens, 1, 8, 4)
    q = rng.standard_normal((1, 2, 8))
    out, lse, _ = oracle.paged_window_decode(q, k, v, table, lens, 0.5, 6, 3)
    t = [0, 1, 2, 24, 25, 26, 27, 28, 29]
    rows = lambda c: np.stack([c[table[0, i // 4], i % 4, 0] for i in t])
    for h in range(2):
        o, l = oracle.softmax_attention(q[0, h][None], rows(k), rows(v), 0.5, [9])
        assert np.allclose(out[0, h], o[0]) and np.isclose(lse[0, h], l[0])


def test_unseen_tokens_are_never_read():
    rng = np.random.default_rng(2)
    lens = [40]
    k, v, table = pages(rng, lens, 1, 8, 4)
    keep = oracle.window_tokens(39, 5, 2)
    k2, v2, t2 = np.full_like(k, np.nan), np.full_like(v, np.nan), np.full_like(table, -1)
    for t in keep:
        t2[0, t // 4] = table[0, t // 4]
        k2[table[0, t // 4], t % 4], v2[table[0, t // 4], t % 4] = k[table[0, t // 4], t % 4], v[table[0, t // 4], t % 4]
    q = rng.standard_normal((1, 1, 8))
    a = oracle.paged_window_decode(q, k, v, table, lens, 1.0, 5, 2)
    b = oracle.paged_window_decode(q, k2, v2, t2, lens, 1.0, 5, 2)
    assert (a[0] == b[0]).all() and (a[1] == b[1]).all()


def test_spans_visit_each_seen_token_once(tmp_path):
    """The units of a windowed decode (host code of the header that the kernels use): each token that the
    query sees is in one unit and not hidden, the others that the units hold are hidden; no unit is idle;
    parts of the units make up the whole."""
    src = tmp_path / "spans.cu"
    src.write_text(r'''
#include "%s/decode_items.cuh"
#include <cstdio>
#include <vector>
namespace metis { int fail(int code, const char*, ...) { return code; }
int encode_tiled(CUtensorMap*, CUtensorMapDataType, int, const void*, const uint64_t*, const uint64_t*, const uint32_t*,
                 CUtensorMapSwizzle, CUtensorMapL2promotion) { return 0; } }
using namespace metis;
int main() {
  const int lens[] = {1, 2, 15, 16, 17, 31, 32, 33, 47, 48, 49, 64, 100, 129, 200};
  const int wins[] = {1, 2, 15, 16, 17, 33, 64, 100, 1000, 0x7fffffff};
  const int sinks[] = {0, 1, 3, 15, 16, 17, 40, 99, 500, 0x7fffffff};
  long checked = 0;
  for (int L : lens) for (int W : wins) for (int K : sinks) {
    const WindowSpan w = window_span(L, W, K);
    std::vector<int> count(L + 64, 0);
    for (int u = 0; u < w.units(); ++u) {
      bool some = false;
      for (int i = 0; i < 16; ++i) {
        const int t = w.token(u) + i;
        if (t < w.t1 && !w.hidden(t)) { ++count[t]; some = true; }
      }
      if (!some) { std::printf("idle unit L %%d W %%d K %%d\n", L, W, K); return 1; }
    }
    int seen = 0;
    for (int t = 0; t < L; ++t) {
      const bool sees = (long)t > (long)L - 1 - W || t < K;
      seen += sees;
      if (count[t] != (sees ? 1 : 0)) { std::printf("L %%d W %%d K %%d t %%d: %%d\n", L, W, K, t, count[t]); return 1; }
    }
    if (w.end() - w.begin() != seen) return 2;
    for (int i = w.begin(); i < w.end(); ++i) if (!count[w.nth(i)] || (i > w.begin() && w.nth(i) <= w.nth(i - 1))) return 3;
    for (int parts = 1; parts <= 8; ++parts) {
      int next = 0;
      for (int p = 0; p < parts; ++p) {
        WindowSpan x = w;
        if (!x.take(p, parts)) continue;
        for (int u = 0; u < x.units(); ++u, ++next) if (x.token(u) != w.token(next)) return 4;
      }
      if (next != w.units()) return 5;
    }
    ++checked;
  }
  const WindowSpan big = window_span(0x7fffffff, 100, 20);
  if (big.token(big.units() - 1) + 15 != 0x7fffffff) return 6;
  std::printf("%%ld\n", checked);
  return 0;
}''' % CSRC)
    exe = tmp_path / "spans"
    r = subprocess.run(["nvcc", "-std=c++17", "--expt-relaxed-constexpr", "-gencode", "arch=compute_103a,code=sm_103a",
                        str(src), "-o", str(exe)], capture_output=True, text=True)
    assert r.returncode == 0, r.stderr[-2000:]
    r = subprocess.run([str(exe)], capture_output=True, text=True)
    assert r.returncode == 0 and int(r.stdout) == 1500, (r.returncode, r.stdout)
