"""Decode on the 4-bit cache over the whole range of its values and scores: small and large values, groups and
rows far apart in size, a dominating key (a sink) over a long tail, parameters written by hand.  Tolerances are
relative to the values, so that small ones count as much as large ones."""

import numpy as np
import pytest
import torch

from oracle import window as W
from tests._lib import built_lib

pytestmark = pytest.mark.gpu

cp_ = None
U16 = 2.0 ** -11  # half a step of fp16, relative
UB = 2.0 ** -8    # half a step of bf16


def setup_module(_):
    global cp_
    if not torch.cuda.is_available():
        pytest.skip("needs a GPU")
    built_lib()
    from context_causal_attention_load_gb300 import cpattn
    cp_ = cpattn


def f64(t):
    return t.detach().double().cpu().numpy()


def _bf16(x):
    return f64(torch.from_numpy(np.asarray(x, np.float32)).to(torch.bfloat16))


def _terms(q, k, v, lens, window, sinks):
    """out, and what its errors are relative to: the sums of P * scale * code and of P * |zero|, and the largest
    sum of |q| (|scale| code + |zero|) / sqrt(D) of a head.  k, v: (codes, scales, zeros)."""
    kv, vv = W.int4_values(*k), W.int4_values(*v)
    want, _ = W.gqa_decode_window(q, kv, vv, lens, window, sinks)
    kabs = W.int4_values(k[0], np.abs(k[1]), np.abs(k[2]))
    code = W.int4_values(v[0], np.abs(v[1]), np.zeros_like(v[2]))
    zero = W.int4_values(np.zeros_like(v[0]), v[1], np.abs(v[2]))
    _, mag_c = W.gqa_decode_window(q, kv, code, lens, window, sinks)
    _, mag_z = W.gqa_decode_window(q, kv, zero, lens, window, sinks)
    B, Hq, D = q.shape
    G = Hq // kv.shape[1]
    smag = np.zeros((B, Hq, 1))
    big = np.zeros((B, Hq, 2, D))  # largest |scale| and |zero| a head sees, per channel
    rows_most = 1
    for b in range(B):
        rows = W.visible_rows(int(lens[b]), window, sinks)
        rows_most = max(rows_most, len(rows))
        if not rows:
            continue
        for h in range(Hq):
            smag[b, h] = (kabs[b, h // G, rows] @ np.abs(q[b, h])).max() / np.sqrt(D)
            for i in (0, 1):
                big[b, h, i] = np.repeat(np.abs(v[1 + i][b, h // G, rows].astype(np.float64)).max(axis=0), 32)
    return want, mag_c, mag_z, smag, big, rows_most


def _tolerance(terms, D):
    """UB: the result's rounding.  U16: P rounded to fp16, and P * scale again.  Of P and of the sum of the P's,
    2^-20 for exp and D * 2^-23 of the scores' magnitude for a score in fp32.  Below fp16's least normal a rounding
    is 2^-25 at most: P is held times 2^14 (2^-39 a row), a scale over a power of two that is at most twice its
    group's largest (2^-24 of that one, weighed with P; the product again 2^-39 a row), codes are 15 at most, and
    where all of a group's scales are below 2^-14 that is the power."""
    want, mag_c, mag_z, smag, big, n = terms
    ep = 2 * (D * 2.0 ** -23 * smag + 2.0 ** -20)
    ceil = np.maximum(2 * big[:, :, 0], 2.0 ** -14)
    sub = n * 2.0 ** -39 * (15 * ceil + big[:, :, 1]) + 15 * 2.0 ** -24 * big[:, :, 0]
    return UB * np.abs(want) + (1 + 2.0 ** -9) * U16 * (2 * mag_c + mag_z) + ep * (mag_c + mag_z) + sub


def _check(q, k, v, lens, window=None, sinks=0):
    """q fp64 [B,Hq,D] (bf16 values), k, v (codes, scales, zeros)"""
    D, Smax = q.shape[2], k[0].shape[2]
    cache = [torch.from_numpy(x).cuda() for t in (k, v) for x in (W.int4_pack(t[0]), W.int4_params(t[1], t[2]))]
    qd = torch.from_numpy(q).to(torch.bfloat16).cuda()
    got = f64(cp_.gqa_decode_int4(qd, *cache, torch.tensor(lens, dtype=torch.int32).cuda(), window, sinks))
    cp_.check_device()
    terms = _terms(q, k, v, lens, Smax if window is None else window, sinks)
    err, tol = np.abs(got - terms[0]), _tolerance(terms, D)
    assert (err <= tol).all(), "worst element at %.2f of its tolerance, off by %.3g of the output's norm" % (
        float((err / tol).max()), float(np.linalg.norm(err) / np.linalg.norm(terms[0])))
    return got


def _rows(rng, B, Hkv, S, D, std, mean=0.0):
    return _bf16(std * (rng.standard_normal((B, Hkv, S, D)) + mean))


# (B, Hq, Hkv, D, Smax, window, sinks): clusters and even shares of all units, one and two tiles of heads
SHAPES = [
    (2, 8, 2, 128, 700, 700, 0),
    (2, 6, 3, 64, 1500, 1000, 4),
    (1, 12, 1, 128, 900, 600, 2),
    (1, 4, 1, 128, 9000, 9000, 0),
    (2, 10, 1, 64, 5000, 4900, 4),
]


def _lens(shape):
    return [shape[4], max(1, shape[4] // 3)][:shape[0]]


@pytest.mark.parametrize("power", [0, 4, 7, 10, 13])
@pytest.mark.parametrize("shape", SHAPES)
def test_values_of_every_size(shape, power):
    """values times 2^-power, scores of standard deviation 2: the tail carries much of the weight"""
    B, Hq, Hkv, D, Smax, window, sinks = shape
    rng = np.random.default_rng(power)
    q = _bf16(2 * rng.standard_normal((B, Hq, D)))
    k = W.int4_quantise(_rows(rng, B, Hkv, Smax, D, 1.0))
    v = W.int4_quantise(_rows(rng, B, Hkv, Smax, D, 2.0 ** -power, 0.5))
    _check(q, k, v, _lens(shape), window, sinks)


@pytest.mark.parametrize("above", [8.0, 11.0, 14.0])
@pytest.mark.parametrize("std", [0.1, 0.01, 0.001])
@pytest.mark.parametrize("shape", SHAPES)
def test_a_sink_over_small_values(shape, std, above):
    """the first key scores `above` over the rest and its own value is small"""
    B, Hq, Hkv, D, Smax, window, sinks = shape
    rng = np.random.default_rng(int(above))
    u = np.sign(rng.standard_normal(D))
    q = _bf16(u + 0.3 * rng.standard_normal((B, Hq, D)))
    k = _rows(rng, B, Hkv, Smax, D, 0.5)
    k[:, :, 0] = _bf16(u * above / np.sqrt(D))
    v = _rows(rng, B, Hkv, Smax, D, std, 0.5)
    v[:, :, 0] *= 2.0 ** -5
    _check(q, W.int4_quantise(k), W.int4_quantise(v), _lens(shape), window, sinks)


@pytest.mark.parametrize("order", ["growing", "falling", "mixed", "groups", "loud row"])
@pytest.mark.parametrize("shape", SHAPES)
def test_rows_and_groups_far_apart(shape, order):
    """scales that grow or fall along the cache, that jump from row to row, and groups 2^20 apart: each group is
    right by its own size"""
    B, Hq, Hkv, D, Smax, window, sinks = shape
    rng = np.random.default_rng(3)
    q = _bf16(rng.standard_normal((B, Hq, D)))
    k = W.int4_quantise(_rows(rng, B, Hkv, Smax, D, 1.0))
    v = _rows(rng, B, Hkv, Smax, D, 1.0, 0.5)
    t = np.arange(Smax)
    if order == "growing":
        v *= np.exp2(np.round(-13 + 16 * t / Smax))[:, None]
    elif order == "falling":
        v *= np.exp2(np.round(3 - 16 * t / Smax))[:, None]
    elif order == "mixed":
        v *= np.exp2(rng.integers(-12, 4, Smax))[:, None]
    elif order == "groups":
        v *= np.repeat(np.exp2(np.linspace(13, -7, D // 32)), 32)
    else:
        v *= 2.0 ** -8
        v[:, :, Smax // 2] *= 2.0 ** 16
    _check(q, k, W.int4_quantise(_bf16(v)), _lens(shape), window, sinks)


@pytest.mark.parametrize("D", [64, 128])
def test_largest_values(D):
    """values at the cache's limit, and scales up to fp16's largest, below zero, subnormal and zero by hand"""
    B, Hq, Hkv, Smax = 1, 4, 2, 300
    rng = np.random.default_rng(7)
    q = _bf16(rng.standard_normal((B, Hq, D)))
    k = W.int4_quantise(_rows(rng, B, Hkv, Smax, D, 1.0))
    _check(q, k, W.int4_quantise(_bf16(57344.0 * np.sign(rng.standard_normal((B, Hkv, Smax, D))))), [Smax])
    codes, _, _ = W.int4_quantise(_rows(rng, B, Hkv, Smax, D, 1.0))
    scale = np.exp2(rng.uniform(-24, 15.9, (B, Hkv, Smax, D // 32)))
    scale *= np.where(rng.random(scale.shape) < 0.3, -1.0, 1.0)
    scale[:, :, 5] = 65504.0
    scale[:, :, 7] = 0.0
    zero = rng.standard_normal(scale.shape)
    _check(q, k, (codes, scale.astype(np.float16), zero.astype(np.float16)), [Smax])
    small = np.ldexp(rng.integers(0, 1024, scale.shape).astype(np.float64), -24)  # subnormal
    _check(q, k, (codes, small.astype(np.float16), (small / 2).astype(np.float16)), [Smax])


@pytest.mark.parametrize("Smax", [200, 4500])
def test_scores_far_apart(Smax):
    """scores of up to 2^22: all the weight on the largest, ties shared"""
    B, Hq, Hkv, D = 1, 2, 1, 128
    rng = np.random.default_rng(9)
    codes, scale, zero = W.int4_quantise(_rows(rng, B, Hkv, Smax, D, 1.0))
    best = [Smax // 3, Smax - 1]
    codes[:] = 0
    codes[:, :, best] = 15
    scale[:] = 1024.0
    zero[:] = -4096.0
    q = np.full((B, Hq, D), 32.0)
    q[:, 1] = -32.0
    v = W.int4_quantise(_rows(rng, B, Hkv, Smax, D, 1.0))
    qd = torch.from_numpy(q).to(torch.bfloat16).cuda()
    cache = [torch.from_numpy(x).cuda() for t in ((codes, scale, zero), v) for x in (W.int4_pack(t[0]), W.int4_params(t[1], t[2]))]
    got = f64(cp_.gqa_decode_int4(qd, *cache, torch.tensor([Smax], dtype=torch.int32).cuda()))
    val = W.int4_values(*v)[0, 0]
    rest = np.delete(val, best, axis=0)
    # equal scores are equal bit for bit, so the weights are: what is left are the roundings of the result, of P * scale
    # and of sums of up to Smax terms in fp32
    code, z = W.int4_values(v[0], v[1], np.zeros_like(v[2]))[0, 0], W.int4_values(np.zeros_like(v[0]), v[1], np.abs(v[2]))[0, 0]
    tol = UB * np.abs(val).max() + (U16 + Smax * 2.0 ** -23) * (code.max() + z.max())
    assert (np.abs(got[0, 0] - val[best].mean(axis=0)) <= tol).all()
    assert (np.abs(got[0, 1] - rest.mean(axis=0)) <= tol).all()
    cp_.check_device()


@pytest.mark.parametrize("Smax", [200, 4500])
@pytest.mark.parametrize("which", ["scale", "zero", "both"])
def test_a_group_that_is_not_a_number(Smax, which):
    """NaN parameters of one group of one row's value: NaN in that group's channels and right everywhere else"""
    B, Hq, Hkv, D = 1, 4, 2, 128
    rng = np.random.default_rng(11)
    q = _bf16(rng.standard_normal((B, Hq, D)))
    k = W.int4_quantise(_rows(rng, B, Hkv, Smax, D, 1.0))
    codes, scale, zero = W.int4_quantise(_rows(rng, B, Hkv, Smax, D, 0.01))
    terms = _terms(q, k, (codes, scale, zero), [Smax], Smax, 0)
    row = Smax // 2
    bs, bz = scale.copy(), zero.copy()
    if which != "zero":
        bs[0, 1, row, 2] = np.nan
    if which != "scale":
        bz[0, 1, row, 2] = np.nan
    codes[0, 1, row, 64:96] = 1
    cache = [torch.from_numpy(x).cuda() for t in (k, (codes, bs, bz)) for x in (W.int4_pack(t[0]), W.int4_params(t[1], t[2]))]
    got = f64(cp_.gqa_decode_int4(torch.from_numpy(q).to(torch.bfloat16).cuda(), *cache,
                                  torch.tensor([Smax], dtype=torch.int32).cuda()))
    cp_.check_device()
    bad = np.zeros(got.shape, bool)
    bad[0, 2:, 64:96] = True
    assert np.isnan(got[bad]).all()
    assert (np.abs(got - terms[0]) <= _tolerance(terms, D))[~bad].all()


@pytest.mark.parametrize("D", [64, 128])
def test_long_flat_caches(D):
    """hundreds of rows a warp, weights alike: the sums of codes and of zeros grow with the rows and cancel.  Rounding
    the exact result to bf16 alone gives an error r; P's and P * scale's rounding to fp16 add some 2^-11 * 0.6 *
    sqrt(1 + (8.7 / 3.7)^2) = 0.0007 to it in quadrature (root mean squares of a uniform rounding, of a code and of a
    value in scales), 9% of r = 0.0016; what adding in fp32 costs has to stay within the same again"""
    B, Hkv, G, Smax = 6, 8, 2, 131072
    g = torch.Generator(device="cuda").manual_seed(13)
    cache = cp_.int4_cache(B, Hkv, Smax, D)
    start = torch.zeros(B, dtype=torch.int32, device="cuda")
    for t0 in range(0, Smax, 32768):
        k, v = (torch.randn(B, 32768, Hkv, D, generator=g, device="cuda").bfloat16() for _ in range(2))
        cp_.kv_append_int4(k, v, start + t0, *cache)
    del k, v
    q = torch.randn(B, Hkv * G, D, generator=g, device="cuda").bfloat16()
    lens = torch.full((B,), Smax, dtype=torch.int32, device="cuda")
    got = cp_.gqa_decode_int4(q, *cache, lens)
    cp_.check_device()
    order = torch.tensor([W._nibble(D, ch) for ch in range(D)], device="cuda")

    def values(codes, params):
        n = torch.stack([codes & 15, codes >> 4], -1).flatten(-2)[..., order].double().unflatten(-1, (D // 32, 32))
        return (n * params[..., 0, :].double()[..., None] + params[..., 1, :].double()[..., None]).flatten(-2)

    want = torch.empty(q.shape, dtype=torch.float64, device="cuda")
    for b in range(B):
        for h in range(Hkv):
            kk, vv = values(cache[0][b, h], cache[1][b, h]), values(cache[2][b, h], cache[3][b, h])
            w = torch.softmax(q[b, h * G:(h + 1) * G].double() @ kk.T / D ** 0.5, -1)
            want[b, h * G:(h + 1) * G] = w @ vv
    err, r = (got.double() - want).norm(), (want.bfloat16().double() - want).norm()
    assert err <= 1.18 * r, float(err / r)
