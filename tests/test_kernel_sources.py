"""Rules of ordering that no run shows reliably, held to the kernels' sources."""
import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "paged_attention_kv_decode_gb300", "csrc")


def source(name):
    with open(os.path.join(CSRC, name)) as f:
        return re.sub(r"//[^\n]*", "", f.read())  # without comments


@pytest.mark.parametrize("name,kernel", [("decode.cu", "decode_rows_beside_kernel"),
                                         ("decode_fp8.cu", "decode_fp8_rows_beside_kernel")])
def test_persistent_decodes_fence_the_ring_between_items(name, kernel):
    """The combine step's ordinary stores and the next item's TMA loads write the same shared memory:
    every thread orders its stores before accesses of the async proxy, in front of the barrier."""
    body = re.search(r"\n\s+" + kernel + r"\(.*?\n}\n", source(name), re.S).group(0)
    loop = body[body.index("for (;;)"):]
    assert "combine_and_store" in loop or "decode_bf16_item" in loop
    assert loop.index("fence_proxy_async_smem();") < loop.index("gsync();")


READ_ONLY = re.compile(r"__ldg\s*\(|\.nc\.|__restrict__")


@pytest.mark.parametrize("name", sorted(f for f in os.listdir(CSRC) if f.endswith((".cu", ".cuh"))))
def test_dependent_kernels_read_with_ordinary_loads(name):
    """A kernel that may start while the one in front runs (it calls pdl_wait) reads nothing through the
    read-only path, which the compiler may also take for `const __restrict__` parameters: caches, index
    arrays and partials may be what the kernel in front writes."""
    text = source(name)
    if name in ("cache_write.cu", "prefix_cache.cu"):  # some of their kernels are launched behind complete ones only
        text = "\n".join(k for k in re.findall(r"__global__.*?\n}\n", text, re.S) if "pdl_wait" in k)
    assert not READ_ONLY.search(text), READ_ONLY.search(text).group(0)


def test_the_chunk_kernel_waits_or_fences_before_it_reads():
    """Beside decodes the chunk kernel's launch, not a wait of its own, orders it behind the kernels that
    write its tables and scales."""
    body = re.search(r"prefill_bf16_kernel\(.*?\n}\n", source("prefill.cu"), re.S).group(0)
    head = body[:body.index("__syncthreads();")]
    assert "if (!p.wait_at_exit) pdl_wait();" in head
    # the warps from 8 on (producers, converters, unit fetcher), but for the one that allocates TMEM
    assert re.search(r"else if \(warp >= 8 && p\.wait_at_exit\) {\s+__threadfence\(\);", head)
