"""Windowed attention over long sequences at head dim 64, alone and with the memory system busy with another
stream's copies: against float64 on the GPU, and the same bit for bit (dq, whose sums' order varies, nearly)."""

import math

import pytest
import torch

from tests._lib import built_lib

pytestmark = pytest.mark.gpu

cp_ = None


def setup_module(_):
    global cp_
    if not torch.cuda.is_available():
        pytest.skip("needs a GPU")
    built_lib()
    from context_causal_attention_load_gb300 import cpattn
    cp_ = cpattn


def _dense(q, k, v, dout, window, sinks):
    """out, lse and gradients in natural order, one head at a time in float64"""
    B, S, Hq, D = q.shape
    G = Hq // k.shape[2]
    p = torch.arange(S, device="cuda")
    see = (p[None] <= p[:, None]) & ((p[:, None] - p[None] < window) | (p[None] < sinks))
    out, lse = torch.empty(q.shape, dtype=torch.float64, device="cuda"), torch.empty(B, Hq, S, dtype=torch.float64, device="cuda")
    dq, dk, dv = (torch.zeros(x.shape, dtype=torch.float64, device="cuda") for x in (q, k, v))
    for b in range(B):
        for h in range(Hq):
            qq, kk, vv, do = q[b, :, h].double(), k[b, :, h // G].double(), v[b, :, h // G].double(), dout[b, :, h].double()
            s = (qq @ kk.T / math.sqrt(D)).masked_fill_(~see, -math.inf)
            lse[b, h] = torch.logsumexp(s, 1)
            w = torch.exp(s - lse[b, h][:, None])
            out[b, :, h] = w @ vv
            ds = w * (do @ vv.T - (do * out[b, :, h]).sum(1, keepdim=True)) / math.sqrt(D)
            dq[b, :, h] = ds @ kk
            dk[b, :, h // G] += ds.T @ qq
            dv[b, :, h // G] += w.T @ do
    return out, lse, dq, dk, dv


@pytest.mark.parametrize("Hq,Hkv,D,S,window,sinks", [(4, 4, 64, 6144, 1024, 4), (6, 2, 64, 5000, 400, 130), (4, 2, 128, 6144, 1024, 4)])
def test_step_under_load(Hq, Hkv, D, S, window, sinks):
    g = torch.Generator(device="cuda").manual_seed(5)
    q, dout = (torch.randn(1, S, Hq, D, generator=g, device="cuda").bfloat16() for _ in range(2))
    k, v = (torch.randn(1, S, Hkv, D, generator=g, device="cuda").bfloat16() for _ in range(2))

    def step():
        out, lse = cp_.attn_fwd_window(q, k, v, 1, window, sinks, False)
        return (out, lse) + tuple(cp_.attn_bwd_window(q, k, v, out, lse, dout, 1, window, sinks, False))

    first = step()
    cp_.check_device()
    for name, a, w in zip(("out", "lse", "dq", "dk", "dv"), first, _dense(q, k, v, dout, window, sinks)):
        # P, dS and the results are rounded to bf16: 2^-8 at most each, some 2^-9 in the norm
        assert (a.double() - w).norm() <= 1e-2 * w.norm(), name
    src, dst = (torch.empty(1 << 29, dtype=torch.uint8, device="cuda") for _ in range(2))
    streams = [torch.cuda.Stream() for _ in range(3)]
    torch.cuda.synchronize()
    runs = []
    for _ in range(12):
        for s in streams[1:]:
            with torch.cuda.stream(s):
                dst.copy_(src)
        with torch.cuda.stream(streams[0]):
            runs.append(step())
    torch.cuda.synchronize()
    cp_.check_device()
    for r in runs:
        for i in (0, 1, 3, 4):
            assert torch.equal(r[i], first[i])
        # fp32 sums in another order, then one rounding
        assert (r[2].float() - first[2].float()).norm() <= 2e-3 * first[2].float().norm()
