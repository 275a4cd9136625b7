"""The smooth activations far out on the negative side, where the values are tiny: relative to themselves, which the
tolerances of the layer's other tests, absolute in |z|, do not see.

Bounds, counted from the arithmetic.  An exponential of q has its argument rounded: q is a constant times z or z^2, two
products (2^-24 each) and the constant's own half step (2^-25), so |q| 2.5 2^-24, at most |q| 2^-22.6, relative in the
result; the hardware's exponential and reciprocal add 2^-22 and 2^-23, the few further products and additions 2^-24
each: 2^-20 together.  The normal distribution's tail adds its fit, 1.6e-5."""
import math

import pytest
import torch

from nvfp4_bit_block_amax_b200 import nvfp4 as N
from tests.test_gpu_layer import F64, bf16, ok, quant_args

pytestmark = pytest.mark.gpu

def ndtr(z):
    """torch's own cancels in 1 + erf below about -5; erfc does not."""
    return torch.special.erfc(-z / math.sqrt(2)) / 2


def layer(M, bias, act):
    Nn = bias.numel()
    a = N.quantize_1d(bf16(M, 64, seed=1))
    b = N.quantize_1d(torch.zeros(Nn, 64, device="cuda", dtype=torch.bfloat16))
    c = N.gemm_epilogue(*quant_args(a), *quant_args(b), M, Nn, 64, bias=bias, activation=act,
                        out_dtype=N.NVFP4_OUT_F32)
    ok()
    return c.to(F64)


def exponent(act, z):
    """|q|, in natural units, of the exponential that the activation rests on."""
    if act == N.NVFP4_ACT_GELU:
        return z * z / 2
    if act == N.NVFP4_ACT_SILU:
        return z.abs()
    return (2 * math.sqrt(2 / math.pi) * (z + 0.044715 * z ** 3)).abs()


def points(act, lo):
    z = torch.linspace(lo, -3, 523, device="cuda").bfloat16()
    return z[exponent(act, z.to(F64)) < 86]          # behind it 2^-126 is near, and results become zeros


def relative(act, z):
    fit = 1.6e-5 if act == N.NVFP4_ACT_GELU else 0.0
    # gelu (tanh) has one product and one sum more in its argument
    return fit + exponent(act, z) * 2.0 ** (-22 if act == N.NVFP4_ACT_GELU_TANH else -22.6) + 2.0 ** -20


@pytest.mark.parametrize("M", [3, 20, 100, 200])
@pytest.mark.parametrize("act,lo", [(N.NVFP4_ACT_GELU, -13), (N.NVFP4_ACT_GELU_TANH, -12), (N.NVFP4_ACT_SILU, -86)])
def test_values(M, act, lo):
    z = points(act, lo)
    # tanh cancels in 1 + tanh(u): through the logistic instead
    z64 = z.to(F64)
    want = z64 * ndtr(z64) if act == N.NVFP4_ACT_GELU else z64 * torch.sigmoid(-exponent(act, z64))
    off = (layer(M, z, act) - want).abs() / want.abs()
    assert (off <= relative(act, z64)).all(), (off / relative(act, z64)).max().item()


@pytest.mark.parametrize("pad", [0, 1])              # whole groups of eight columns, and single ones
@pytest.mark.parametrize("act,lo", [(N.NVFP4_ACT_GELU, -12), (N.NVFP4_ACT_GELU_TANH, -9), (N.NVFP4_ACT_SILU, -80)])
def test_slopes(act, lo, pad):
    """In binary32, as the bias gradient of a single row."""
    z = points(act, lo)
    n = z.numel() // 8 * 8 - pad * 3
    z = z[:n]
    row = torch.zeros(1, (n + 7) // 8 * 8, device="cuda").bfloat16()
    row[0, :n] = z
    _, db = N.act_grad(torch.ones_like(row)[:, :n], row[:, :n], act)
    ok()
    z = z.to(F64)
    if act == N.NVFP4_ACT_GELU:
        dens = z * torch.exp(-z * z / 2) / math.sqrt(2 * math.pi)
        want, parts = ndtr(z) + dens, ndtr(z) + dens.abs()
    else:
        s = torch.sigmoid(-exponent(act, z))
        dx = 1.0 if act == N.NVFP4_ACT_SILU else 2 * math.sqrt(2 / math.pi) * (1 + 3 * 0.044715 * z * z)
        want, parts = s + z * s * (1 - s) * dx, s + (z * s * dx).abs()
    # each part has the tail's relative error; they partly cancel
    assert ((db.to(F64) - want).abs() <= parts * relative(act, z)).all()


def test_gelu_stored_in_bf16_is_rounded_right():
    """A stored gelu is off by bf16's half step, 2^-8 of the value at most (8 significant bits), and by a hundredth of
    another: 3e-5 / 2^-8 for the value itself."""
    z = points(N.NVFP4_ACT_GELU, -12)
    a = N.quantize_1d(bf16(200, 64, seed=1))
    b = N.quantize_1d(torch.zeros(z.numel(), 64, device="cuda", dtype=torch.bfloat16))
    want = z.to(F64) * ndtr(z.to(F64))
    for M in (3, 200):
        c = N.gemm_epilogue(a.codes[:M], a.scales_mma, a.global_scale, *quant_args(b), M, z.numel(), 64, bias=z,
                            activation=N.NVFP4_ACT_GELU)
        ok()
        assert ((c.to(F64) - want).abs() <= want.abs() * 1.01 * 2.0 ** -8).all()
