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


def test_the_notes_of_a_windows_unit_are_cleared_before_it_is_published():
    """A unit without a partial tile waits for nothing that the warp which notes V rows does: bits that its
    slot still held, or memory that nothing had written, would add tokens to its rows."""
    text = source("prefill.cu")
    fetcher = text[text.index("warp == kMmaWarp + 2"):text.index("WINDOW && warp > kMmaWarp")]
    publish = fetcher.index("unit_info[slot] = it")
    assert fetcher.index("wait_all(&unit_empty") < fetcher.index("xw.odd[slot][lane] = 0u") < publish
    assert fetcher.index("xw.any_odd[slot] = 0") < publish
    guard = text[text.index("WINDOW && warp > kMmaWarp"):]
    guard = guard[:guard.index("softmax groups") if "softmax groups" in guard else guard.index("regs_inc")]
    assert "any_odd[slot] = 0" not in guard and "odd[slot][lane]" not in guard


def test_every_cta_counts_the_tokens_in_whole_numbers():
    """Each CTA of the kernel over the prefixes works out for itself how many share them: a sum of fp32 that
    threads add up in any order rounds differently from CTA to CTA beyond 2^24 tokens."""
    text = source("prefill.cu")
    body = text[text.index("int pf_shared_ctas("):text.index("PfShare pf_share(")]
    assert "atomicAdd" not in body and "long long tokens = -shared_tokens" in body
    assert not re.search(r"float\s+(shared_)?tokens", text[text.index("int pf_shared_ctas("):text.index("prefill_bf16_kernel(const")])
