"""A first call on the legacy stream while a stream that waits for it is being captured: refused like one inside the
capture, which stays valid."""

import subprocess
import sys

import pytest
import torch

pytestmark = pytest.mark.gpu

CODE = """
import ctypes, torch
from context_causal_attention_load_gb300 import cpattn as c, synth
q, k, v, _ = (x.cuda() for x in synth.attention_inputs(1, 384, 4, 2, 64, 64, seed=3))
out, lse = c.attn_fwd_window(q, k, v, 1, 100, 4, False)
torch.cuda.synchronize()
rt = ctypes.CDLL("libcudart.so.13")
s, g = ctypes.c_void_p(), ctypes.c_void_p()
assert rt.cudaStreamCreate(ctypes.byref(s)) == 0  # (one that waits for the legacy stream)
assert rt.cudaStreamBeginCapture(s, 0) == 0
p = lambda t: ctypes.c_void_p(t.data_ptr())
rc = c.load().cp_attn_fwd_window(p(q), p(k), p(v), p(out), p(lse), 1, 4, 2, 384, 64, 1, 0, 101, 4, None)
msg = c.load().cp_attn_last_error()
assert c.load().cp_attn_fwd_window(p(q), p(k), p(v), p(out), p(lse), 1, 4, 2, 384, 64, 1, 0, 100, 4, s) == 0
assert rt.cudaStreamEndCapture(s, ctypes.byref(g)) == 0 and g.value
assert rc == -1 and b"capture" in msg, (rc, msg)
rt.cudaGraphDestroy(g)
rt.cudaStreamDestroy(s)
again, _ = c.attn_fwd_window(q, k, v, 1, 101, 4, False)
c.check_device()
"""


def test_first_call_beside_a_capture():
    if not torch.cuda.is_available():
        pytest.skip("needs a GPU")
    r = subprocess.run([sys.executable, "-c", CODE], capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stderr[-2000:]
