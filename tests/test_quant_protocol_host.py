"""Orders that the 8-bit cache's kernels keep among their threads, which no run
can show: read from the source (CPU)."""
import os
import re

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))),
                    "rank_kv_cache_lrkv_b200", "csrc")


def _source(name):
    """The file without comments, white space as one blank."""
    with open(os.path.join(CSRC, name)) as f:
        text = re.sub(r"//[^\n]*|/\*.*?\*/", " ", f.read(), flags=re.S)
    return re.sub(r"\s+", " ", text)


def test_an_append_counts_a_cta_after_all_its_warps_have_read_the_length():
    """The CTA that is counted last stores the new length, so a CTA is counted
    behind a barrier that every path of it meets: a late warp would read the
    new length and append the call's tokens a second time."""
    text = _source("quant_cache.cu")
    kernel = text[text.index("quant_append_kernel(QuantAppendArgs a) {"):]
    assert kernel.index("quant_len(c, b)") < kernel.index("atomicAdd(&c.counter[b], 1)")
    before = kernel[:kernel.index("atomicAdd(&c.counter[b], 1)")]
    # nothing but the count's own branch stands between the barrier and it, and
    # the barrier is in no branch: as many braces are open there as at the start
    head, tail = before.rsplit("__syncthreads();", 1)
    assert re.fullmatch(r" if \(tid == 0\) \{ __threadfence\(\); const int last = [^;{}]*; if \(", tail)
    assert head.count("{") - head.count("}") == 1


def test_copies_still_landing_when_a_wait_gave_up_are_waited_for():
    """A CTA may not end with a bulk copy into its shared memory under way.  A
    warp that gives up on a page goes on counting it as read, so what may still
    land are the last slabs asked for, one a stage, read or not; and a role that
    ended well cannot know that another gives up later."""
    helper = _source("quant.cuh")
    body = helper[helper.index("void quant_drain("):]
    assert body.startswith("void quant_drain(uint64_t* bars, int issued, int stages) { "
                           "const uint64_t t0 = global_ns(); "
                           "for (int k = max(0, issued - stages); k < issued; ++k) "
                           "while (!mbar_try_wait(&bars[k % stages], (k / stages) & 1) && "
                           "global_ns() - t0 < ")
    decode, few = _source("quant_decode.cu"), _source("quant_few.cu")
    # a failed wait sets `fail` for the warp that looks at its own slabs here
    assert "if (*fail && warp < W && lane == 0) { quant_drain(bar, n_issued, D);" in decode
    assert re.search(r"\} \} \} \} if \(lane == 0\) quant_drain\(rawfull, issued, NR\); \}", few)
    for text in (decode, few):
        assert text.count("quant_drain(") == 1
