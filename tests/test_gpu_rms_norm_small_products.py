"""RMS norm to 8 bits where the largest |sum weight| of a row is small, or no fp32
number at all, on the GPU.

The bytes are round(t (448 / top)) of fp32 products t, whose mantissas do not depend
on their exponents: the oracle takes exact products in 64 bits, brings the largest
near 1 by a power of two and goes on in fp32, on the CPU.  The scale, top rstd / 448,
carries rstd's error (c of test_gpu_rms_norm.py) and three roundings; a scale below
fp32's normal range is off by a step of 2^-149 too.
"""
import math

import pytest
import torch

import diffusion_transformer_qk_amd as qkr
from tests.test_gpu_layer_norm import DEV, EPS, F, TYPES, C, gen, rows_of
from tests.test_gpu_rms_norm import FP8, summed

pytestmark = pytest.mark.gpu


def oracle(s, w, eps):
    s, w = s.double().cpu(), w.double().cpu()
    t = s * w
    top = t.abs().amax(-1, keepdim=True)
    e = torch.frexp(top).exponent
    t32 = torch.ldexp(t, -e).float()
    top32 = t32.abs().amax(-1, keepdim=True)
    top32 = torch.where(top32 == 0, torch.ones_like(top32), top32)
    q = (t32 * (torch.full_like(top32, 448.0) / top32)).to(FP8)
    rstd = 1 / torch.sqrt(s.square().mean(-1, keepdim=True) + eps)
    return q, (torch.where(top == 0, torch.ones_like(top), top) * rstd / 448).squeeze(-1), (top != 0).squeeze(-1)


def check(x, w, residual=None, eps=EPS):
    found = qkr.rms_norm_fp8(x, w, residual=residual, eps=eps)
    q, scales = found[0].cpu(), found[1].cpu().double()
    want, scale, some = oracle(summed(x, residual), w, eps)
    assert torch.equal(q.view(torch.uint8) & 0x7f, want.view(torch.uint8) & 0x7f)
    nonzero = want.float() != 0
    assert torch.equal(q.view(torch.uint8)[nonzero], want.view(torch.uint8)[nonzero])
    assert bool(torch.isfinite(scales).all()) and bool((scales >= 0).all())
    assert bool(((scales - scale).abs() <= (C + 8 * F) * scale + 2.0 ** -149)[some].all())


HIDDEN = [8, 264, 520, 1024, 1032, 2056, 5120, 8192]


@pytest.mark.parametrize("hidden", HIDDEN)
@pytest.mark.parametrize("dtype,param", [("bf16", "fp32"), ("fp16", "fp32"), ("bf16", "bf16")])
@pytest.mark.parametrize("by", [2.0 ** -95, 2.0 ** -104, 1e-37, 2.0 ** -130, 2.0 ** -140])
def test_small_weights(hidden, dtype, param, by):
    x, r = rows_of(41, 9, hidden, dtype), rows_of(42, 9, hidden, dtype)
    w = ((1 + 0.3 * torch.randn(hidden, generator=gen(43))).double() * by).to(TYPES[param]).to(DEV)
    check(x, w)
    check(x, w, r)


@pytest.mark.parametrize("hidden", HIDDEN)
@pytest.mark.parametrize("x_by,w_by", [(1e-30, 1e-30), (1e-38, 1e-38), (1e-20, 1e-4), (1e30, 1e-38), (1e-39, 1.0),
                                       (1e-35, 1e30)])
def test_small_rows_and_weights(hidden, x_by, w_by):
    x = (rows_of(44, 7, hidden, "bf16").double() * x_by).to(torch.bfloat16)
    w = ((1 + 0.3 * torch.randn(hidden, generator=gen(45))).double() * w_by).float().to(DEV)
    check(x, w)
    check(x, w, eps=1e-30)


@pytest.mark.parametrize("hidden", HIDDEN)
def test_products_of_unlike_factors(hidden):
    """Neither factor is small everywhere, their products are; and rows of zeros between."""
    x = torch.full((5, hidden), 2.0 ** -120, dtype=torch.bfloat16, device=DEV) * (1 + torch.arange(
        hidden, device=DEV) % 7).to(torch.bfloat16)
    w = torch.full((hidden,), 1.5, device=DEV)
    x[:, hidden // 2] = 3.0
    w[hidden // 2] = 2.0 ** -121
    x[1] = x[3] = 0
    x[4] *= -1
    check(x, w)
    w[hidden // 2] = 0
    check(x, w)
    x[:, hidden // 2] = 0
    check(x, w)
    # products of zero alone, of rows that are not zeros
    check(torch.ones_like(x), torch.zeros_like(w))


def test_rows_of_nan_alone():
    for hidden in HIDDEN:
        x = torch.zeros((3, hidden), dtype=torch.bfloat16, device=DEV)
        x[1] = math.nan
        q, scales = qkr.rms_norm_fp8(x, torch.full((hidden,), 1e-38, device=DEV))
        assert bool(torch.isnan(scales[1])) and bool(torch.isfinite(scales[::2]).all())
        assert bool((q[::2].float() == 0).all())
        assert bool(torch.isnan(qkr.rms_norm(x)[1]).all())


@pytest.mark.parametrize("hidden", HIDDEN)
def test_scales_of_infinite_rows(hidden):
    """NaN, whatever weight an infinity meets: 0 makes its product NaN, which no maximum sees."""
    x = torch.ones((4, hidden), dtype=torch.bfloat16, device=DEV)
    x[1, 3], x[2, 3] = math.inf, -math.inf
    for value in (0.0, -0.0, 1e-38, 1.0, math.nan):
        w = torch.ones(hidden, device=DEV)
        w[3] = value
        scales = qkr.rms_norm_fp8(x, w)[1]
        assert bool(torch.isnan(scales[1:3]).all()) and bool(torch.isfinite(scales[::3]).all())
