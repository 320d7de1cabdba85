"""16-bit results of the orthogonalised updates: what fp32 results are, rounded once."""

import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


@pytest.fixture(scope="module")
def muon():
    from block_wise_dynamic_gb300 import build

    build.build()
    from block_wise_dynamic_gb300 import muon as m

    return m


def draw(rows, cols, seed, kind):
    rng = np.random.default_rng(seed)
    g = rng.standard_normal((rows, cols))
    if kind == "strong":  # a few directions far above the rest
        r = max(1, min(rows, cols) // 32)
        g = 0.02 * g + rng.standard_normal((rows, r)) @ rng.standard_normal((r, cols))
    return torch.from_numpy(1e-3 * g).to(DEV)


# few tiles, whose steps all run on the matrix itself; and more, of sides too near each other for steps among the squares
SHAPES = [(40, 70), (300, 300), (301, 777), (64, 1000), (1000, 1000), (1500, 1600), (1100, 900)]


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("shape", SHAPES)
def test_direct_steps_round_once(muon, shape, dtype):
    """The same 16-bit values in fp32 take the same products, so that the results are the same before they are rounded."""
    for kind in ("gauss", "strong"):
        for steps in (1, 5):
            g = draw(*shape, 1, kind).to(dtype)
            assert torch.equal(muon.orthogonalize(g, steps), muon.orthogonalize(g.float(), steps).to(dtype))


def test_steps_round_once(muon):
    """The step too: from zeros and without momentum a parameter becomes the update."""
    for shape in ((300, 200), (64, 1000), (900, 1000)):
        g = draw(*shape, 2, "strong").to(torch.bfloat16)
        got = []
        for kind in (torch.bfloat16, torch.float32):
            p, m = torch.zeros(shape, dtype=kind, device=DEV), torch.zeros(shape, device=DEV)
            muon.MuonArgs([p], [g], [m]).step(lr=1.0, momentum=0.0, nesterov=False)
            got.append(p)
        assert torch.equal(got[0], got[1].to(torch.bfloat16))


@pytest.mark.parametrize("shape", [(1320, 1650), (1600, 2048), (1100, 2100)])
def test_up_to_two_columns_to_a_row_round_once(muon, shape):
    """The steps run on the matrix itself up to there."""
    g = draw(*shape, 3, "strong").to(torch.bfloat16)
    assert torch.equal(muon.orthogonalize(g), muon.orthogonalize(g.float()).to(torch.bfloat16))


def test_results_repeat(muon):
    """The same bits each time, whatever ran before in the same memory."""
    for shape, dtype in (((2816, 1024), torch.bfloat16), ((1000, 2100), torch.float32), ((1500, 1600), torch.bfloat16), ((301, 777), torch.float32)):
        g, other = draw(*shape, 4, "strong").to(dtype), draw(*shape, 5, "gauss").to(dtype)
        first = muon.orthogonalize(g)
        for _ in range(5):
            muon.orthogonalize(other)
            assert torch.equal(muon.orthogonalize(g), first)


def test_last_products_with_an_added_matrix_repeat(muon):
    """Large tiles whose last product adds the matrix that it multiplies, in both orientations: the same bits each time."""
    for shape in ((1500, 2300), (2300, 1500)):
        for dtype in (torch.float32, torch.bfloat16, torch.float16):
            g = draw(*shape, 6, "strong").to(dtype)
            first = muon.orthogonalize(g)
            assert all(torch.equal(muon.orthogonalize(g), first) for _ in range(20))
