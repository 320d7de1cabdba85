"""AdamW with fp32 moments over lists of tensors, and the gradients' norm and
clipping factor, against the 64-bit statements in ``oracle.adamw32``."""

import numpy as np
import pytest
import torch

from oracle import adamw32 as ref

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
TYPES = {"fp32": torch.float32, "bf16": torch.bfloat16, "fp16": torch.float16}
ROUND = {"fp32": 2.0 ** -24, "bf16": 2.0 ** -8, "fp16": 2.0 ** -11}
TINY = {"fp32": 0.0, "bf16": 0.0, "fp16": 2.0 ** -25}
HP = dict(lr=1e-3, beta1=0.9, beta2=0.999, eps=1e-8, weight_decay=0.01)


@pytest.fixture(scope="module")
def bwd():
    from block_wise_dynamic_gb300 import build

    build.build()
    import block_wise_dynamic_gb300 as m

    return m


def np64(t):
    return t.double().cpu().numpy()


def tensors(sizes, kind, seed, std, offset=0):
    """Views of one buffer, each starting `offset` elements past a multiple of 64."""
    g = torch.Generator(DEV).manual_seed(seed)
    out = []
    for n in sizes:
        buf = torch.randn(n + 64, generator=g, device=DEV) * std
        out.append(buf.to(TYPES[kind])[offset:offset + n])
    return out


def state(sizes, pk, gk, seed, offset=0):
    p, g = tensors(sizes, pk, seed, 0.02, offset), tensors(sizes, gk, seed + 1, 1e-3, offset)
    m = tensors(sizes, "fp32", seed + 2, 3e-4, offset)
    v = [t.square() if offset == 0 else t.square_() for t in tensors(sizes, "fp32", seed + 3, 1e-3, offset)]
    return p, g, m, v


def check(old, new, pk, step, scale=1.0):
    for i in range(len(new[0])):
        p, g, m, v = (np64(t) for t in (old[0][i], old[1][i], old[2][i], old[3][i]))
        b1, b2 = HP["beta1"], HP["beta2"]
        rp, rm, rv = ref.step(p, g, m, v, **HP, step=step, scale=scale)
        gs = np.abs(g * scale)
        # m: a coefficient, a product and a sum (and g'), half a unit each; v: one product more
        assert np.all(np.abs(np64(new[2][i]) - rm) <= 4 * 2.0 ** -24 * (b1 * np.abs(m) + (1 - b1) * gs) + 1e-44)
        assert np.all(np.abs(np64(new[3][i]) - rv) <= 6 * 2.0 ** -24 * (b2 * np.abs(v) + (1 - b2) * gs * gs) + 1e-44)
        # the update: m's error (of the size of its terms), and ten roundings of the quotient; then p's own
        terms = (b1 * np.abs(m) + (1 - b1) * gs) / (np.abs(rm) + 1e-300)
        update = np.abs(rp - p * (1 - HP["lr"] * HP["weight_decay"]))
        bound = update * 2.0 ** -24 * (4 * terms + 12) + 3 * 2.0 ** -24 * (np.abs(p) + update) + ROUND[pk] * np.abs(rp) + TINY[pk] + 1e-40
        assert np.all(np.abs(np64(new[0][i]) - rp) <= bound)


LISTS = [[1], [5, 2048, 2049, 3], [4096 * 3 + 7], [1, 0, 70001], [100] * 1000]


@pytest.mark.parametrize("gk", ["fp32", "bf16", "fp16"])
@pytest.mark.parametrize("pk", ["fp32", "bf16", "fp16"])
@pytest.mark.parametrize("sizes", LISTS, ids=lambda s: f"{len(s)}x{max(s)}")
def test_step(bwd, sizes, pk, gk):
    old = state(sizes, pk, gk, 1)
    new = [[t.clone() for t in ts] for ts in old]
    bwd.adam32_step_multi(*new, **HP, step=3)
    check(old, new, pk, 3)
    assert all(torch.equal(a, b) for a, b in zip(old[1], new[1]))


@pytest.mark.parametrize("offset", [1, 2, 3])
@pytest.mark.parametrize("pk,gk", [("fp32", "fp32"), ("bf16", "bf16"), ("fp16", "fp32")])
def test_step_unaligned(bwd, offset, pk, gk):
    sizes = [5000, 2048, 9]
    new = state(sizes, pk, gk, 2, offset)
    old = [[t.clone() for t in ts] for ts in new]
    args = bwd.MultiTensorArgs32(*new)
    args.step(**HP, step=1)
    check(old, new, pk, 1)


@pytest.mark.parametrize("offsets", [(1, 2, 3, 0), (0, 0, 0, 1), (3, 3, 3, 7), (5, 1, 9, 13)])
@pytest.mark.parametrize("pk,gk", [("fp32", "fp32"), ("bf16", "fp16")])
def test_step_arrays_that_start_differently(bwd, offsets, pk, gk):
    sizes = [1, 2, 3, 1023, 1024, 1025, 5000]
    new = [tensors(sizes, pk, 31, 0.02, offsets[0]), tensors(sizes, gk, 32, 1e-3, offsets[1]),
           tensors(sizes, "fp32", 33, 3e-4, offsets[2]), [t.square_() for t in tensors(sizes, "fp32", 34, 1e-3, offsets[3])]]
    whole = [[t._base.clone() for t in ts] for ts in new]
    old = [[t.clone() for t in ts] for ts in new]
    bwd.adam32_step_multi(*new, **HP, step=2)
    check(old, new, pk, 2)
    for k, ts in enumerate(new):  # nothing beside the tensors is written
        for t, w in zip(ts, whole[k]):
            w[offsets[k]:offsets[k] + t.numel()] = t
            assert torch.equal(t._base, w)


def test_step_reads_the_factor_on_the_device(bwd):
    old = state([3000, 17], "fp32", "bf16", 3)
    new = [[t.clone() for t in ts] for ts in old]
    args = bwd.MultiTensorArgs32(*new)
    factor = torch.full((1,), 0.25, device=DEV)
    args.step(**HP, step=7, grad_scale=factor)
    check(old, new, "fp32", 7, 0.25)
    kept = [[t.clone() for t in ts] for ts in new]
    for bad in (float("nan"), float("inf"), -float("inf")):
        factor.fill_(bad)
        args.step(**HP, step=8, grad_scale=factor)
    assert all(torch.equal(a, b) for x, y in zip(kept, new) for a, b in zip(x, y))


def test_non_finite_gradient_stays_in_its_element(bwd):
    old = state([3000], "fp32", "fp32", 4)
    old[1][0][1234] = float("nan")
    new = [[t.clone() for t in ts] for ts in old]
    bwd.adam32_step_multi(*new, **HP, step=2)
    for k in (0, 2, 3):
        bad = ~torch.isfinite(new[k][0])
        assert bad[1234] and int(bad.sum()) == 1


def test_new_gradients_in_an_old_table(bwd):
    old = state([100, 4000], "fp32", "bf16", 5)
    new = [[t.clone() for t in ts] for ts in old]
    args = bwd.MultiTensorArgs32(*new)
    other = tensors([100, 4000], "bf16", 77, 1e-3)
    args.set_grads(other)
    args.step(**HP, step=1)
    check([old[0], other, old[2], old[3]], new, "fp32", 1)


@pytest.mark.parametrize("gk", ["fp32", "bf16", "fp16"])
@pytest.mark.parametrize("sizes", LISTS + [[3] * 2500, [2048 * 4000 + 1]], ids=lambda s: f"{len(s)}x{max(s)}")
@pytest.mark.parametrize("offset", [0, 1, 3, 6])
def test_norm(bwd, sizes, gk, offset):
    g = tensors(sizes, gk, 6, 1e-2, offset)
    for max_norm, loss_scale in ((0.01, 1.0), (1e9, 1.0), (0.5, 1024.0), (float("inf"), 3.0)):
        factor, norm = bwd.GradNorm(g).clip_scale(max_norm, loss_scale)
        rf, rn = ref.clip([np64(t) for t in g], max_norm, loss_scale)
        # at most 2,048 * 4,001 / (152 * 256) = 211 fp32 additions per thread, here fewer: 256 half units
        np.testing.assert_allclose(float(norm), rn, rtol=256 * 2.0 ** -24)
        np.testing.assert_allclose(float(factor), rf, rtol=256 * 2.0 ** -24)


def test_norm_is_deterministic_and_reusable(bwd):
    g = tensors([300_001] * 5, "bf16", 8, 1.0)
    handle = bwd.GradNorm(g)
    first = [float(t) for t in handle.clip_scale(1.0)]
    for _ in range(20):
        assert [float(t) for t in handle.clip_scale(1.0)] == first
    assert int(handle._work[:16].sum()) == 0


def test_norm_of_nothing_and_of_non_finite_values(bwd):
    factor, norm = bwd.GradNorm([], device=DEV).clip_scale(1.0)
    assert float(norm) == 0.0 and float(factor) == 1.0
    for bad in (float("nan"), float("inf")):
        g = tensors([5000, 10], "fp32", 9, 1.0)
        g[1][3] = bad
        factor, norm = bwd.clip_scale(g, 1.0)
        assert torch.isnan(factor).all() and not torch.isfinite(norm).any()


def test_clipped_step_end_to_end(bwd):
    old = state([3000, 17], "fp32", "bf16", 10)
    new = [[t.clone() for t in ts] for ts in old]
    factor, _ = bwd.clip_scale(new[1], 0.01)
    bwd.adam32_step_multi(*new, **HP, step=2, grad_scale=factor)
    check(old, new, "fp32", 2, float(factor))


def test_refusals(bwd):
    p, g, m, v = state([10, 20], "fp32", "bf16", 11)
    with pytest.raises(ValueError):
        bwd.MultiTensorArgs32(p, g[:1], m, v)
    with pytest.raises(TypeError):
        bwd.MultiTensorArgs32(p, [g[0], g[1].float()], m, v)
    with pytest.raises(TypeError):
        bwd.MultiTensorArgs32(p, g, [t.half() for t in m], v)
    with pytest.raises(ValueError):
        bwd.MultiTensorArgs32(p, g, [m[0], m[1][:5]], v)
    with pytest.raises(ValueError):
        bwd.MultiTensorArgs32([t.cpu() for t in p], g, m, v)
    args = bwd.MultiTensorArgs32(p, g, m, v)
    for kw in (dict(step=0), dict(step=1, eps=-1.0), dict(step=1, beta1=1.0), dict(step=1, weight_decay=-0.1)):
        with pytest.raises(bwd.BwdError):
            args.step(**kw)
    with pytest.raises(TypeError):
        args.step(step=1, grad_scale=torch.ones(1, device=DEV, dtype=torch.float64))
    with pytest.raises(ValueError):
        args.step(step=1, grad_scale=torch.ones(2, device=DEV))
    with pytest.raises(TypeError):
        args.set_grads([t.float() for t in g])
    norm = bwd.GradNorm(g)
    for max_norm, loss_scale in ((0.0, 1.0), (-1.0, 1.0), (float("nan"), 1.0), (1.0, 0.0), (1.0, float("inf"))):
        with pytest.raises(bwd.BwdError):
            norm.clip_scale(max_norm, loss_scale)
    with pytest.raises(ValueError):
        bwd.GradNorm([])
