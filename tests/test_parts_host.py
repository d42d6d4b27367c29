"""The tolerance of fp32 products in three bf16 parts lies between what the scheme leaves out and what a lost product of parts costs (no GPU needed)."""
import pytest
import torch

from _parts import LEFT_OUT, TERMS, product, rms, tolerance


@pytest.fixture(scope="module")
def factors():
    g = torch.Generator().manual_seed(1)
    return torch.randn(200, 512, generator=g), torch.randn(512, 300, generator=g)


def test_the_six_products(factors):
    a, b = factors
    exact = a.double() @ b.double()
    assert rms(product(a, b) - exact) <= LEFT_OUT * rms(exact)


@pytest.mark.parametrize("lost", TERMS)
def test_a_lost_product_is_seen(factors, lost):
    a, b = factors
    exact = a.double() @ b.double()
    off = rms(product(a, b, [t for t in TERMS if t != lost]) - exact) / rms(exact)
    # the largest tolerances in use: sums of up to 2048 terms, of two products of up to 640
    assert off > 1.5 * max(tolerance(2048), tolerance(640, pairs=2))


@pytest.mark.parametrize("wrong", [((1, 1), (1, 2), (2, 0), (0, 1), (1, 0), (0, 0)), ((1, 1), (0, 2), (0, 2), (0, 1), (1, 0), (0, 0))])
def test_a_wrong_part_is_seen(factors, wrong):
    a, b = factors
    exact = a.double() @ b.double()
    assert rms(product(a, b, wrong) - exact) > 1.5 * tolerance(2048) * rms(exact)
