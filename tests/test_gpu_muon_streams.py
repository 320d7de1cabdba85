"""Workspaces of the optimizer step on other streams than the one they were made on, and in graphs."""

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


def draw(shape, seed):
    return torch.from_numpy(np.random.default_rng(seed).standard_normal(shape).astype(np.float32)).to(DEV)


def lists(seed):
    shapes = [(300, 500), (500, 300)]
    return [draw(s, seed + i) for i, s in enumerate(shapes)], [draw(s, seed + 10 + i) for i, s in enumerate(shapes)], [torch.zeros(s, device=DEV) for s in shapes]


def busy(stream):
    """Some milliseconds of work on a stream."""
    with torch.cuda.stream(stream):
        a = torch.ones(6000, 6000, device=DEV)
        for _ in range(3):
            a = a @ a * 1e-4
    return a


@pytest.mark.parametrize("how", ["argument", "current", "handle"])
def test_a_dropped_list_keeps_its_workspace_until_the_step_has_run(muon, how):
    """The step waits behind other work on a side stream while the list's memory is handed out and written."""
    busy(torch.cuda.current_stream())  # libraries set up
    ps, gs, ms = lists(1)
    twin = [[t.clone() for t in l] for l in (ps, gs, ms)]
    muon.MuonArgs(*twin).step()
    torch.cuda.synchronize()
    torch.cuda.empty_cache()
    side = torch.cuda.Stream()
    args = muon.MuonArgs(ps, gs, ms)
    size = args.work.numel()
    torch.cuda.synchronize()
    kept = busy(side)
    if how == "argument":
        args.step(stream=side)
    elif how == "handle":
        args.step(stream=side.cuda_stream)
    else:
        with torch.cuda.stream(side):
            args.step()
    running = not side.query()
    del args
    others = [torch.full((size,), 255, dtype=torch.uint8, device=DEV) for _ in range(4)]
    assert running
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(ps + ms, twin[0] + twin[2]))
    del kept, others


def test_a_graph_keeps_its_workspace(muon):
    """Replayed after the optimizer's plan, and with it the list's workspace, was replaced, and that memory written."""
    ps, gs, _ = lists(3)
    params = [[torch.nn.Parameter(ps[0].clone()), torch.nn.Parameter(draw((700, 900), 30))] for _ in range(2)]
    grads = [gs[0], draw((700, 900), 31)]
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        one, two = (muon.Muon(p) for p in params)
        params[0][0].grad = grads[0]
        one.step()
        graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph, stream=side):
        one.step()
    with torch.cuda.stream(side):
        params[0][1].grad = grads[1]
        one.step()  # a new plan, whose workspace is larger
        others = [torch.full((1 << 20,), 255, dtype=torch.uint8, device=DEV) for _ in range(40)]
        graph.replay()
        # the same three steps: of one matrix, of both (which divides the sums in another way), and of one
        for both in (False, True, False):
            params[1][0].grad, params[1][1].grad = grads[0], grads[1] if both else None
            two.step()
    torch.cuda.synchronize()
    assert torch.equal(params[0][0], params[1][0]) and torch.equal(params[0][1], params[1][1])
    del others


def test_an_optimizer_on_a_side_stream(muon):
    """Steps on another stream than the first one's, whose plan and workspace are replaced while they wait."""
    torch.cuda.empty_cache()
    side = torch.cuda.Stream()
    ps, gs, _ = lists(2)
    a, b = ([torch.nn.Parameter(p.clone()) for p in ps] for _ in range(2))
    one, two = muon.Muon(a), muon.Muon(b)
    for opt, params, stream in ((one, a, side), (two, b, torch.cuda.current_stream())):
        params[0].grad = gs[0]
        opt.step()  # one matrix, on the current stream
        torch.cuda.synchronize()
        params[1].grad = gs[1]
        with torch.cuda.stream(stream):
            kept = busy(stream)
            opt.step()  # both: a new plan
            opt.step()
            params[1].grad = None
            opt.step()  # another
        torch.empty(1 << 24, dtype=torch.uint8, device=DEV).fill_(255)
        torch.cuda.synchronize()
        del kept
    assert all(torch.equal(p, q) for p, q in zip(a, b))


def test_a_limited_workspace(muon):
    """Fewer matrices at a time; a copied optimizer and one that resumes keep the limit, and it can be changed between steps."""
    import copy

    from oracle import muon as ref

    shapes = [(300, 700)] * 9 + [(40, 60), (30, 90)]
    gs = [draw(s, 50 + i) for i, s in enumerate(shapes)]
    want = [-0.1 * 0.2 * max(s) ** 0.5 * ref.orthogonalize(g.double().cpu().numpy()) for s, g in zip(shapes, gs)]

    def near(params):
        for p, w in zip(params, want):
            # beside an error of some 20 bits, what 300 times the truth's rounding in fp32 leaves
            assert np.linalg.norm(p.detach().double().cpu().numpy() - w) <= 300 * 2.0 ** -24 * np.linalg.norm(w)

    sizes = []
    for limit in (None, 8 << 20, 1):
        ps, ms = [torch.zeros(s, device=DEV) for s in shapes], [torch.zeros(s, device=DEV) for s in shapes]
        args = muon.MuonArgs(ps, gs, ms, work_bytes=limit)
        args.step(lr=0.1)
        near(ps)
        sizes.append(args.work.numel())
    assert sizes[0] > 8 << 20 >= sizes[1] > sizes[2]

    params = [torch.nn.Parameter(torch.zeros(s, device=DEV)) for s in shapes]
    opt = muon.Muon(params, lr=0.1, work_bytes=8 << 20)
    for p, g in zip(params, gs):
        p.grad = g
    opt.step()
    near(params)
    assert [w.numel() for w in opt._work.values()] == [sizes[1]]
    assert copy.deepcopy(opt).param_groups[0]["work_bytes"] == 8 << 20
    state = opt.state_dict()
    del state["param_groups"][0]["work_bytes"]  # as an earlier version saved it
    opt.load_state_dict(state)
    opt.step()
    assert sizes[0] in [w.numel() for w in opt._work.values()]
    opt.param_groups[0]["work_bytes"] = 1
    opt.step()
    assert all(p.isfinite().all() for p in params)


def test_a_list_has_one_workspace(muon):
    """Made by its first step, on that one's stream: a list made elsewhere holds no second one."""
    ps, gs, ms = lists(4)
    torch.cuda.synchronize()
    torch.cuda.empty_cache()
    before = torch.cuda.memory_allocated()
    side = torch.cuda.Stream()
    args = muon.MuonArgs(ps, gs, ms)
    assert torch.cuda.memory_allocated() == before
    for _ in range(3):
        args.step(stream=side)
        assert torch.cuda.memory_allocated() - before == (args.work.numel() + 511) // 512 * 512
    # captured first: the graph's own, and then one for the list
    other = muon.MuonArgs(*[[t.clone() for t in l] for l in (ps, gs, ms)])
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        other.step()
    twin = [[t.clone() for t in l] for l in (ps, gs, ms)]
    graph.replay()
    other.step()
    again = muon.MuonArgs(*twin)
    again.step()
    again.step()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(twin[0], other._keep[0]))


def test_an_optimizer_whose_first_step_is_captured(muon):
    ps, gs, _ = lists(5)
    a, b = ([torch.nn.Parameter(p.clone()) for p in ps] for _ in range(2))
    for params in (a, b):
        for p, g in zip(params, gs):
            p.grad = g
    muon.orthogonalize(gs[0])
    one, two = muon.Muon(a), muon.Muon(b)
    for p in a:  # state that outlives the graph's memory
        one.state[p]["momentum_buffer"] = torch.zeros_like(p)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        one.step()
    graph.replay()
    one.step()
    graph.replay()
    for _ in range(3):
        two.step()
    torch.cuda.synchronize()
    assert all(torch.equal(p, q) for p, q in zip(a, b))


def test_a_first_step_that_is_captured_is_refused(muon):
    """Each replay would start from no momentum."""
    ps, gs, _ = lists(6)
    params = [torch.nn.Parameter(p) for p in ps]
    params[0].grad = gs[0]
    opt = muon.Muon(params)
    graph = torch.cuda.CUDAGraph()
    with pytest.raises(RuntimeError, match="first step"):
        with torch.cuda.graph(graph):
            opt.step()
    before = [p.detach().clone() for p in params]
    opt.step()
    params[1].grad = gs[1]  # another parameter's first one
    graph = torch.cuda.CUDAGraph()
    with pytest.raises(RuntimeError, match="first step"):
        with torch.cuda.graph(graph):
            opt.step()
    opt.step()
    torch.cuda.synchronize()
    assert all(p.isfinite().all() and not torch.equal(p, b) for p, b in zip(params, before))
