"""The 4-bit attention brings a share of the next projections' weights into L2 with each CTA of its grid."""
import os
import re

SRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "speculative_decoding_verify_step_gb300", "csrc",
                   "kv4_attention.cu")


def test_ctas_without_a_piece_prefetch_their_share_too():
    """Shares are cut by the grid, which may have more CTAs than there are pieces: one that returns early, with
    nothing to attend to, brings its share, and does so after the wait for its predecessor."""
    text = re.sub(r"//[^\n]*", "", open(SRC).read())
    kernel = text[text.index("kv4_attention_kernel("):text.index("kv4_merge_kernel(")]
    early = kernel[kernel.index(">= plan.total"):]
    early = early[:early.index("return;")]
    assert early.index("pdl_wait()") < early.index("prefetch_next()")
    share = kernel[kernel.index("prefetch_next ="):]
    share = share[:share.index("};")]
    assert share.count("l2_prefetch_share(p.l2_next[") == 2
    assert kernel.count("prefetch_next()") == 2               # one for each way through the kernel
