"""The windowed calls' work lists: any number of shapes takes a bounded amount of memory, a shape whose list has gone
answers as before, and captured graphs keep theirs."""

import ctypes

import pytest
import torch

from context_causal_attention_load_gb300 import cpattn, synth
from tests._lib import built_lib


def test_workspace_sizes_kept_are_bounded(monkeypatch):
    asked = []

    def run(name, dev, *args):
        asked.append(args[:-1])
        args[-1]._obj.value = 0

    monkeypatch.setattr(cpattn, "_run", run)
    monkeypatch.setattr(cpattn, "_ws_bytes", {})
    for i in range(20000):
        assert cpattn._workspace("query", 0, (1, i), None) == (None, 0)
        assert len(cpattn._ws_bytes) <= 4096
    n = len(asked)
    cpattn._workspace("query", 0, (1, 19999), None)
    assert len(asked) == n


def _grown(before):
    torch.cuda.synchronize()
    return before - torch.cuda.mem_get_info()[0]


@pytest.mark.gpu
def test_any_number_of_shapes():
    if not torch.cuda.is_available():
        pytest.skip("needs a GPU")
    lib = built_lib()
    B, S, H, D = 4, 16384, 8, 64
    g = torch.Generator(device="cuda").manual_seed(3)
    q, k, v, dout = (torch.randn(B, S, H, D, generator=g, device="cuda").bfloat16() for _ in range(4))
    out, lse = torch.empty_like(q), torch.empty(B, H, S, device="cuda")

    def fwd(w):
        return cpattn.attn_fwd_window(q, k, v, 1, w, 0, False, out=out, lse=lse)

    # a small step of each kind, eager and captured
    small = [x.cuda() for x in synth.attention_inputs(1, 640, 4, 2, 64, 64, seed=9)]

    def step():
        o, l = cpattn.attn_fwd_window(*small[:3], 1, 77, 2, False)
        return [o, l] + list(cpattn.attn_bwd_window(*small[:3], o, l, small[3], 1, 77, 2, False))

    want = [x.clone() for x in step()]
    first = [x.clone() for x in fwd(1)]
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = step()
    before = torch.cuda.mem_get_info()[0]
    n = ctypes.c_size_t(0)
    for w in range(2, 1002):  # 1000 lists of 64 KB forward, and of 64 KB and more backward
        fwd(w)
        assert lib.cp_attn_bwd_window_workspace(B, H, H, S, D, 1, 0, w, 0, ctypes.byref(n), None) == 0
    # 16 MB each, and the pieces device memory comes in
    assert _grown(before) <= 40 << 20, _grown(before)
    same = lambda a, b: all(torch.equal(a[i], b[i]) for i in (0, 1, 3, 4))  # noqa: E731  (dq's sums vary in order)
    graph.replay()
    torch.cuda.synchronize()
    assert same(got, want) and same(step(), want)
    assert all(torch.equal(a, b) for a, b in zip(fwd(1), first))
    # a list that has gone is a first call again: not inside a capture, and after one outside
    gr = torch.cuda.CUDAGraph()
    with torch.cuda.graph(gr):
        fwd(1)
        with pytest.raises(cpattn.CpAttnError, match="capture"):
            fwd(2)
    gr.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, first[0])
    fwd(2)
    cpattn.check_device()
