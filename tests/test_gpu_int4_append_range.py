"""Rows quantised into the 4-bit cache, bit for bit, over the whole range of bf16: from groups below fp16's least
scale (where zeros and scales are subnormal and coarse) to clamped ones, and values that lie on and next to ties."""

import numpy as np
import pytest
import torch

from oracle import window as W
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


def _same(x):
    """x bf16 [T, Hkv, D]: what the cache holds after an append of it, against the oracle"""
    T, Hkv, D = x.shape
    cache = cp_.int4_cache(1, Hkv, T, D)
    start = torch.zeros(1, dtype=torch.int32, device="cuda")
    xs = x[None].cuda()
    cp_.kv_append_int4(xs, -xs, start, *cache)
    cp_.check_device()
    for y, codes, params in ((x, *cache[:2]), (-x, *cache[2:])):
        c, s, z = W.int4_quantise(y.double().numpy().transpose(1, 0, 2))
        assert np.array_equal(params[0].cpu().numpy(), W.int4_params(s, z), equal_nan=True)
        wrong = codes[0].cpu().numpy() != W.int4_pack(c)
        assert not wrong.any(), "%d bytes of %d" % (wrong.sum(), wrong.size)


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("power", list(range(-30, -12)) + [-8, -1, 0, 5, 11, 14, 15, 16, 17, 60])
def test_every_magnitude(power, D):
    g = torch.Generator().manual_seed(1000 + power)
    x = torch.randn(1024, 2, D, generator=g) * 2.0 ** power
    _same(x.to(torch.bfloat16))


@pytest.mark.parametrize("power", [-26, -24, -22, -20, -18, -15, -3, 0, 3])
def test_ties_and_their_neighbours(power):
    """groups whose span is 15 steps of a power of two, with values half a step (and a little more or less) from
    whole ones, and a least value that fp16 holds or not"""
    D, T = 128, 1024
    g = torch.Generator().manual_seed(2000 + power)
    step = 2.0 ** power
    n = torch.randint(0, 31, (T, 1, D // 32, 32), generator=g) / 2.0
    n[..., 0], n[..., 1] = 0.0, 15.0
    n[..., 4:] += (torch.randint(-1, 2, n[..., 4:].shape, generator=g) * 2.0 ** -7).clamp(-0.5, 0.5)
    base = (torch.randint(-20, 20, (T, 1, D // 32, 1), generator=g) / 4.0)
    x = ((n + base) * step).reshape(T, 1, D)
    _same(x.to(torch.bfloat16))


def test_mixed_groups():
    """groups of all sizes beside one another, some with a few values of another size"""
    g = torch.Generator().manual_seed(5)
    T, D = 4096, 128
    x = torch.randn(T, 1, D // 32, 32, generator=g) * torch.exp2(torch.randint(-28, 16, (T, 1, D // 32, 1), generator=g).float())
    few = torch.rand(x.shape, generator=g) < 0.1
    x = torch.where(few, x * torch.exp2(torch.randint(-12, 3, x.shape, generator=g).float()), x)
    x[::7] = x[::7].abs() + x[::7].abs().amax(-1, keepdim=True) * 3  # far from zero
    _same(x.reshape(T, 1, D).to(torch.bfloat16))


@pytest.mark.parametrize("power", [-23, -20, -14, -7, 0, 6, 11])
def test_values_far_smaller_than_their_group(power):
    """zeros half a step from a whole code, and values so much smaller that a difference in fp32 does not show them:
    which side of the tie they lie on decides; groups with a clamped value among them"""
    D, T = 128, 1024
    g = torch.Generator().manual_seed(3000 + power)
    half = torch.randint(0, 15, (T, 1, D // 32, 1), generator=g) + 0.5
    tiny = torch.exp2(-torch.randint(18, 46, (T, 1, D // 32, 32), generator=g).float())
    x = tiny * torch.randint(-1, 2, tiny.shape, generator=g)
    x[..., 0], x[..., 1] = -half[..., 0], 15.0 - half[..., 0]
    x = x * 2.0 ** power
    if power == 11:
        x[::2, ..., 1] = 1e6
    _same(x.reshape(T, 1, D).to(torch.bfloat16))


def test_scales_on_and_beside_ties():
    """spans of 15 * (2m + 1) / 2 of fp16's least scale, and a hair more or less"""
    D, T = 128, 512
    g = torch.Generator().manual_seed(4000)
    m = torch.randint(0, 8, (T, 1, D // 32, 1), generator=g)
    x = torch.zeros(T, 1, D // 32, 32)
    x[..., 5] = (15 * (2 * m + 1))[..., 0] * 2.0 ** -25
    x[..., 9] = (torch.randint(-1, 2, (T, 1, D // 32), generator=g) * torch.exp2(-torch.randint(45, 60, (T, 1, D // 32), generator=g).float()))
    x[..., 10:] = x[..., 5:6] * torch.randint(0, 17, (T, 1, D // 32, 22), generator=g) / 16
    low = x[..., 9] > 0
    x[..., :5] = torch.where(low[..., None], x[..., 9:10], x[..., :5])  # no zeros below a least value above zero
    x[..., 6:9] = torch.where(low[..., None], x[..., 9:10], x[..., 6:9])
    x[..., 10:] = torch.maximum(x[..., 10:], x[..., 9:10])
    _same(x.reshape(T, 1, D).to(torch.bfloat16))
