"""What the memory model asks of the kernels' source where running cannot show it."""

import os
import re

from tests._lib import ROOT


def test_launch_control_answers_are_read_before_they_are_asked_for_again():
    """the answer is written by the async proxy, read by the generic one, and its bytes are written again: a proxy
    fence stands between the read and what follows it"""
    src = open(os.path.join(ROOT, "context_causal_attention_load_gb300", "csrc", "common.cuh")).read()
    body = re.search(r"int clc_answer\(.*?^}\n", src, flags=re.S | re.M).group(0)
    read, fence = body.index("w[1]"), body.find("fence_proxy_async_smem()")
    assert fence > read
