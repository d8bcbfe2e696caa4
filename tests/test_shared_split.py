"""The count of SMs for shared prefixes, compiled for the host from the kernels' own header."""
import os
import subprocess

import pytest

from paged_attention_kv_decode_gb300 import build as builder

SMS = 152


@pytest.fixture(scope="module")
def count(tmp_path_factory):
    """count(cases of (tiles, units, bytes of own tokens)): the CTAs that each takes."""
    at = tmp_path_factory.mktemp("split")
    src, exe = at / "split.cu", at / "split"
    src.write_text('#include <stdio.h>\n#include "' + os.path.join(builder.CSRC, "shared_split.cuh") + '"\n'
                   "using namespace metis;\nint main() {\n  int tiles, units, sms;\n  float bytes;\n"
                   '  while (scanf("%d %d %f %d", &tiles, &units, &bytes, &sms) == 4) {\n'
                   "    unsigned long long best = ~0ull;\n"
                   "    for (int n = 1; n <= shared_split_most(bytes, sms); ++n) {\n"
                   "      const unsigned long long key = shared_split_key(tiles, units, bytes, n, sms);\n"
                   "      if (key < best) best = key;\n    }\n"
                   '    printf("%d\\n", (int)(unsigned)best);\n  }\n}\n')
    subprocess.run([builder.nvcc(), *builder.ARCH, "-std=c++17", str(src), "-o", str(exe)], check=True, capture_output=True)

    def run(cases):
        ask = "".join("%d %d %.9g %d\n" % (*c, SMS) for c in cases)
        r = subprocess.run([str(exe)], input=ask, text=True, capture_output=True, check=True)
        return [int(x) for x in r.stdout.split()]
    return run


def model(tiles, units, own, n):
    prefix = 7 + 2 * -(-tiles // n) + 5 * -(-units // n)
    return max(prefix, 7 + own / min(40e3 * (SMS - n), 6.1e6) if n < SMS else 0.0)


CASES = [(1, 1, 0.0), (1, 1, 1e6), (8, 8, 0.0), (1024, 8, 8e7), (1280, 256, 4e8), (200, 100, 1e3), (5000, 8, 1e9),
         (10 ** 6, 1000, 1e8), (19 * 10 ** 6, 200, 1e6), (30 * 10 ** 6, 8192, 4e10), (2 ** 31 - 1, 2 ** 20, 0.0),
         (2 ** 31 - 1, 2 ** 31 - 1, 1e10), (600 * 10 ** 6, 10 ** 6, 2e11)]


def test_the_count_is_the_cheapest_however_long_the_work(count):
    """Within the sixteenth of a microsecond in which times are compared, and fp32's rounding of them."""
    for case, n in zip(CASES, count(CASES)):
        most = SMS - 1 if case[2] > 0 else SMS
        assert 1 <= n <= most
        best = min(model(*case, m) for m in range(1, most + 1))
        assert model(*case, n) <= best * (1 + 2.0 ** -20) + 1 / 16, (case, n)


def test_much_shared_work_takes_nearly_every_sm(count):
    assert all(n >= SMS - 2 for n in count([(t, 200, 1e6) for t in (10 ** 6, 19 * 10 ** 6, 2 ** 31 - 1)]))
