"""Uses of the caches and their pages that change something between calls: settings behind a recorded step, rows that
pause, pages that rows share, calls that are refused half-way."""
import pytest
import torch

import adaptive_sparse_hierarchical_b200 as D

pytestmark = pytest.mark.gpu

HQ, HKV, DIM, B, PAGE = 8, 2, 64, 32, 64


def _ints(*v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def _rnd(seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return lambda *s: torch.randn(*s, device="cuda", generator=g).bfloat16()


def _make(batch=3, cap=512, gamma=3.0, **kw):
    qbar = torch.randn(HKV, DIM, device="cuda", generator=torch.Generator(device="cuda").manual_seed(1)) * 0.3
    return D.Q4DecodeState(batch, cap, HQ, HKV, DIM, chunk=B, alpha=1.5, gamma=gamma, page_size=PAGE, qbar=qbar, **kw)


def _step(rnd, batch=3):
    return rnd(batch, HQ, DIM), rnd(batch, HKV, DIM), rnd(batch, HKV, DIM)


def _same_state(a, b):
    for name in ("k_codes", "v_codes", "k_scales", "v_scales", "kbar", "state", "seqlens"):
        assert torch.equal(getattr(a, name), getattr(b, name)), name


def test_a_recorded_step_follows_its_settings():
    """graph_step after qbar, the route outputs or the pools' description changed equals the eager step."""
    rnd = _rnd(2)
    eager, graph = _make(), _make()
    K, V = rnd(3, 100, HKV, DIM), rnd(3, 100, HKV, DIM)
    old = graph.qbar
    for st in (eager, graph):
        st.fill(K, V, [100, 31, 0])
    routes = {id(st): [torch.zeros(3, HKV, dtype=torch.int32, device="cuda") for _ in range(2)] for st in (eager, graph)}

    def run(n):
        for _ in range(n):
            ins = _step(rnd)
            assert torch.equal(eager.step(*ins).clone(), graph.graph_step(*ins))
        _same_state(eager, graph)

    run(3)
    other = torch.randn(HKV, DIM, device="cuda")
    eager.qbar = graph.qbar = other
    run(40)
    for k in range(2):
        for st in (eager, graph):
            st.route = D.route_out(routes[id(st)][k])
        run(40)
        assert torch.equal(routes[id(eager)][k], routes[id(graph)][k]) and routes[id(graph)][k].any()
    first = routes[id(graph)][0].clone()
    assert torch.equal(first, routes[id(eager)][0])
    for st in (eager, graph):
        st.route, st.qbar = None, old
    run(40)
    assert torch.equal(first, routes[id(graph)][0])


def test_a_recording_that_fails_leaves_no_graph(monkeypatch):
    """What was not recorded is not replayed: the next call steps eagerly and records."""
    rnd = _rnd(3)
    eager, graph = _make(), _make()
    a, b = _step(rnd), _step(rnd)
    eager.step(*a), eager.step(*b)
    want = eager.step(*b).clone()

    def fail(*args, **kw):
        raise RuntimeError("no recording")

    with monkeypatch.context() as m:
        m.setattr(torch.cuda, "graph", fail)
        with pytest.raises(RuntimeError, match="no recording"):
            graph.graph_step(*a)
    graph.graph_step(*b)
    assert torch.equal(graph.graph_step(*b), want)
    _same_state(eager, graph)
