"""Shared by the tests of the grouped products: quantized weights, their values
in binary64, and the tolerance of a 16-bit output."""

import torch

from bit_group_wise_amd import q4

DEV = "cuda:0"
ACTS = {q4.F16: torch.float16, q4.BF16: torch.bfloat16}
FORMATS = [q4.NF4, q4.INT4_SYM, q4.INT4_ASYM, q4.NF4_DQ, q4.FP4]


def generator(seed):
    gen = torch.Generator(device=DEV)
    gen.manual_seed(seed)
    return gen


def weight(rows, K, fmt, g, gen):
    w = torch.randn((rows, K), generator=gen, device=DEV) * K ** -0.5
    return q4.quantize(w.half(), fmt, g)


def values(q, act):
    """The weight [rows, K] in binary64, each value rounded to the activations' type."""
    return q4.dequantize(q, ACTS[act]).double()


def normal(gen, act, *shape, size=1.0):
    return (torch.randn(shape, generator=gen, device=DEV) * size).to(ACTS[act])


def half_step(act):
    return torch.finfo(ACTS[act]).eps / 2


def tiny(act):
    """Half the spacing of the smallest values."""
    return 2.0 ** -25 if act == q4.F16 else 2.0 ** -134


def assert_product(got, want, absdot, terms, act, tag=""):
    """`terms` products summed in binary32 and rounded once: each addition is off
    by at most a step of the sum (2^-23, the matrix cores may cut where they do
    not round) relative to the sum of the magnitudes, the rounding by half a
    step of the output's type, which also takes the sum's error in."""
    err = (got.double() - want).abs()
    sums = terms * 2.0 ** -23 * absdot
    tol = sums + half_step(act) * (want.abs() + sums) + tiny(act)
    assert bool(torch.isfinite(got).all()), f"{tag} not finite"
    worst = (err - tol).max()
    assert bool(worst <= 0), f"{tag} off by {float(err.max())}, past the tolerance by {float(worst)}"
