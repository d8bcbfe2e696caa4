"""Rules that no run shows reliably, held to the sources of the kernels over shared prefixes and windows."""
import re

from test_kernel_sources import source


def kernel(name, file):
    return re.search(r"\b" + name + r"\(.*?\n}\n", source(file), re.S).group(0)


def test_a_late_cta_leaves_as_one():
    """The counter of claimed shares changes while a CTA looks at it: one thread decides for all, before
    the barriers that the loads complete on are initialised by another."""
    body = kernel("decode_own_kernel", "shared_prefix.cu")
    head = body[:body.index("mbar_init")]
    returns = head.count("return;")
    assert returns == 1 and re.search(r"if \(__syncthreads_or\(\w+\)\) {\s+pdl_wait\(\);\s+return;", head)
    assert re.search(r"if \(threadIdx\.x == 0\) {[^}]*next_share", head)


def test_the_decodes_of_own_tokens_end_behind_the_prefixes():
    """The join waits for the grid directly in front of it only: that one has to end after the one before it."""
    body = kernel("decode_own_kernel", "shared_prefix.cu")
    assert re.search(r"pdl_wait\(\);\s*}\s*$", body)


def test_the_guard_of_windows_waits_for_every_tile():
    """A wait tells a phase from the next one only: a warp that skips a tile's wait may take the next phase for done."""
    text = source("prefill.cu")
    guard = text[text.index("WINDOW && warp > kMmaWarp"):]
    loop = guard[guard.index("for (int j = 0; j < it.n_kv; ++j, ++t)"):guard.index("xw.v_ready[st]")]
    assert loop.index("wait_all(&v_full[st]") < loop.index("if (!pf_partial(it, j))")
    skipped = loop[loop.index("if (!pf_partial(it, j))"):loop.index("continue;")]
    assert "mbar_arrive(&v_empty[st])" in skipped
