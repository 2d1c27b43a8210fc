"""A shape's first call sets up device memory (work lists, the error word): that memory is complete before any
stream may read it, streams that do not wait for the legacy one among them."""

import os
import re

import pytest
import torch

from context_causal_attention_load_gb300 import synth
from tests._lib import ROOT, built_lib


def test_set_up_memory_is_waited_for():
    """blocking copies from host memory and memsets in the host code stand only where their end is waited for (a copy
    from pageable memory may return once it is staged)"""
    src = open(os.path.join(ROOT, "context_causal_attention_load_gb300", "csrc", "api.cu")).read()
    bodies = re.findall(r"^cudaError_t (copy_to_device|clear_device)\(.*?^}\n", src, flags=re.S | re.M)
    assert sorted(bodies) == ["clear_device", "copy_to_device"]
    rest = src
    for m in re.finditer(r"^cudaError_t (?:copy_to_device|clear_device)\(.*?^}\n", src, flags=re.S | re.M):
        assert "cudaStreamSynchronize(cudaStreamLegacy)" in m.group(0)
        rest = rest.replace(m.group(0), "")
    assert "cudaMemcpyHostToDevice" not in rest and not re.search(r"\bcudaMemset\(", rest)


@pytest.mark.gpu
def test_first_calls_on_a_side_stream():
    if not torch.cuda.is_available():
        pytest.skip("needs a GPU")
    built_lib()
    from context_causal_attention_load_gb300 import cpattn as c
    B, S, Hq, Hkv, D = 1, 2048, 8, 4, 64
    q, k, v, dout = (x.cuda() for x in synth.attention_inputs(B, S, Hq, Hkv, D, D, seed=41))
    busy = torch.empty(1 << 28, dtype=torch.uint8, device="cuda")
    side = torch.cuda.Stream()
    torch.cuda.synchronize()

    def step(window):
        out, lse = c.attn_fwd_window(q, k, v, 1, window, 3, False)
        return [out, lse] + list(c.attn_bwd_window(q, k, v, out, lse, dout, 1, window, 3, False))

    windows = list(range(301, 325))  # (no other test's)
    first = []
    for w in windows:
        busy.zero_()  # the legacy stream has work
        with torch.cuda.stream(side):
            first.append(step(w))
    torch.cuda.synchronize()
    c.check_device()
    for w, got in zip(windows, first):
        again = step(w)
        for i in (0, 1, 3, 4):
            assert torch.equal(got[i], again[i])
        assert (got[2].float() - again[2].float()).norm() <= 2e-3 * again[2].float().norm()
    c.check_device()
