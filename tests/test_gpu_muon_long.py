"""Orthogonalised updates of long rows: no accumulator takes more than 128 products."""

import numpy as np
import pytest
import torch

from oracle import muon as ref

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


@pytest.fixture(scope="module")
def muon():
    from block_wise_dynamic_gb300 import build

    build.build()
    from block_wise_dynamic_gb300 import muon as m

    return m


def np64(t):
    return t.detach().double().cpu().numpy()


def one_step(muon, shape):
    """Error of one step on u v^T, relative to the result: (a + b + c) u v^T / |u v^T|."""
    rng = np.random.default_rng(1)
    g = torch.from_numpy(np.outer(rng.standard_normal(shape[0]), rng.standard_normal(shape[1])).astype(np.float32)).to(DEV)
    want = ref.orthogonalize(np64(g), 1)
    return np.linalg.norm(np64(muon.orthogonalize(g, 1)) - want) / np.linalg.norm(want)


# one matrix of so few tiles that the kernel for those takes its first product, with all of the summed axis to a CTA, or an eighth of it
@pytest.mark.parametrize("shape", [(1408, 32768), (1408, 16384), (130, 60000), (65000, 65)])
def test_one_step_of_a_single_direction(muon, shape):
    """All products of a sum have one sign there, and truncated additions make it smaller by a share t that grows with the
    accumulator's products.  Of the result, with A = u u^T, that is a share |b + 2 c| t = 0.71 t from A, 2.03 t from A A and 2.74 t
    from B X, over a + b + c = 0.701: 7.8 t, and as much from each product however long the rows are, if each accumulator takes the
    same number of products.  So the error is that of a matrix of 2048 x 2048, whose products all go to the kernel for large
    tiles, but for where a sum lies between two powers of two: what an addition cuts off is a fixed part of the lower
    power, and so between a whole and a half of that part of the sum.  Hence at most twice.

    (The bound was 9.7e-7, from 2e-10 for each of 128 products and the roundings of pairs.  That figure does not hold: with 10,944 products to an
    accumulator the error was 6.4e-5, 5.9e-9 for each, and 2048 x 2048 has 1.05e-6.)"""
    off, most = one_step(muon, shape), 2 * one_step(muon, (2048, 2048))
    assert off <= most, (off, most)


def test_long_and_short_rows_together(muon):
    """One launch for both, in which CTAs of the short ones have no stage of the summed axis."""
    rng = np.random.default_rng(2)
    shapes = [(64, 16384), (20, 30), (100, 300), (20, 70)]
    gs = [torch.from_numpy(rng.standard_normal(s).astype(np.float32)).to(DEV) for s in shapes]
    ps, ms = [torch.zeros(s, device=DEV) for s in shapes], [torch.zeros(s, device=DEV) for s in shapes]
    args = muon.MuonArgs(ps, gs, ms)
    args.work.fill_(255)  # NaN wherever nothing was written
    args.step(lr=1.0, momentum=0.0, nesterov=False, rms=1.0)
    for p, g, shape in zip(ps, gs, shapes):
        want = -max(shape) ** 0.5 * ref.orthogonalize(np64(g))
        # beside an error of some 20 bits, what 300 times the truth's rounding in fp32 leaves
        assert np.linalg.norm(np64(p) - want) <= 300 * 2.0 ** -24 * np.linalg.norm(want)


def steps_in_fp32(g):
    a, b, c = 3.4445, -4.7750, 2.0315
    x = g.t() if g.shape[0] > g.shape[1] else g
    x = x / (x.square().sum().sqrt() + 1e-7)
    for _ in range(5):
        gram = x @ x.t()
        x = a * x + (b * gram + c * gram @ gram) @ x
    return x.t() if g.shape[0] > g.shape[1] else x


@pytest.mark.parametrize("shape", [(64, 65536), (30000, 130), (16, 65536), (300, 30000)])
def test_error_of_long_rows(muon, shape):
    """No more than four times that of the same steps in fp32: operands have 22 bits instead of 24."""
    rng = np.random.default_rng(3)
    for strong in (False, True):
        g = rng.standard_normal(shape)
        if strong:
            r = max(1, min(shape) // 4)
            g += (rng.standard_normal((shape[0], r)) * np.exp(-3 * np.arange(r) / r)) @ rng.standard_normal((r, shape[1]))
        g = torch.from_numpy(1e-3 * g).to(DEV, torch.float32)
        want = ref.orthogonalize(np64(g))
        off, plain = (np.linalg.norm(np64(o) - want) / np.linalg.norm(want) for o in (muon.orthogonalize(g), steps_in_fp32(g)))
        assert off <= 4 * plain, (strong, off, plain)


def test_more_than_sixteen_columns_to_a_row_round_once(muon):
    """The steps run on the matrix itself from there on."""
    for shape in ((130, 30000), (17000, 1024)):
        g = torch.from_numpy(np.random.default_rng(4).standard_normal(shape)).to(DEV, torch.bfloat16)
        assert torch.equal(muon.orthogonalize(g), muon.orthogonalize(g.float()).to(torch.bfloat16))


@pytest.mark.parametrize("shape", [(1024, 4096), (1408, 5632), (16384, 1408), (1000, 1000), (301, 777)])
def test_documented_error(muon, shape):
    """8e-6 of a result's norm at most, alone (small tiles for all or some of the products) and four together (large ones for most)."""
    rng = np.random.default_rng(5)
    r = min(shape) // 64
    gs = rng.standard_normal((4, *shape)) + 2 * rng.standard_normal((4, shape[0], r)) @ rng.standard_normal((4, r, shape[1]))
    gs = torch.from_numpy(1e-3 * gs).to(DEV, torch.float32)
    want = ref.orthogonalize(np64(gs[0]))
    for got in (muon.orthogonalize(gs[0]), muon.orthogonalize(gs)[0]):
        assert np.linalg.norm(np64(got) - want) <= 8e-6 * np.linalg.norm(want)
