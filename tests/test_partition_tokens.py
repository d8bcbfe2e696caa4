"""The token range of a partition, compiled for the host from the kernels' own header."""
import os
import subprocess

from paged_attention_kv_decode_gb300 import build as builder

CASES = [(0, 16), (1, 16), (16, 16), (17, 16), (1000, 48), ((1 << 30) + 100, 1 << 30), ((1 << 31) - 1, 1 << 30),
         ((1 << 31) - 1, (1 << 31) - 16), ((1 << 31) - 1, 3 << 29)]


def test_partitions_cover_a_sequence_without_overflow(tmp_path):
    src, exe = tmp_path / "ranges.cu", tmp_path / "ranges"
    src.write_text('#include <stdio.h>\n#include "' + os.path.join(builder.CSRC, "decode.cuh") + '"\n'
                   "int main() {\n  int L, P, part, t0, t1;\n"
                   '  while (scanf("%d %d %d", &L, &P, &part) == 3) {\n'
                   "    metis::partition_tokens(L, P, part, t0, t1);\n"
                   '    printf("%d %d\\n", t0, t1);\n  }\n}\n')
    subprocess.run([builder.nvcc(), *builder.ARCH, "-std=c++17", str(src), "-o", str(exe)], check=True, capture_output=True)
    ask = [(L, P, part) for L, P in CASES for part in range(min(-(-L // P), 50))]
    r = subprocess.run([str(exe)], input="".join("%d %d %d\n" % a for a in ask), text=True, capture_output=True, check=True)
    got = [tuple(map(int, line.split())) for line in r.stdout.splitlines()]
    assert got == [(part * P, min(L, part * P + P)) for L, P, part in ask]
