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
