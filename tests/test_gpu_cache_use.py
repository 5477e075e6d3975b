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


@pytest.mark.parametrize("layers", [1, 2])
def test_fill_spares_pages_that_rows_share(layers):
    """After a fork, fill would write the prompt into pages that another row reads: it changes nothing and check()
    tells why; with the rows freed and pages given out anew it runs, into pages of its own."""
    rnd = _rnd(4)
    table = torch.full((4, 8), -1, dtype=torch.int32, device="cuda")
    sts = [_make(4, num_pages=20, page_table=table) for _ in range(layers)]
    pool = D.PagePool.of(sts)
    K, V, q = rnd(4, 200, HKV, DIM), rnd(4, 200, HKV, DIM), rnd(4, HQ, DIM)
    lens = _ints(200, 70, 0, 0)
    pool.reserve(lens)
    for st in sts:
        st.fill(K, V, lens)
        st.fill(V, K, lens)       # (nothing is shared yet)
        st.fill(K, V, lens)
    pool.fork([0], [3])
    pool.check()
    before = [[t.clone() for t in (st.k_codes, st.v_codes, st.k_scales, st.v_scales, st.kbar, st.state, st.seqlens)] for st in sts]
    out = [st.decode(q).clone() for st in sts]
    for k, st in enumerate(sts):
        for bad in ([150, 0, 0, 0], _ints(0, 0, 0, 150), [200, 70, 0, 200]):
            st.fill(V, K, bad)
            for x, y in zip(before[k], (st.k_codes, st.v_codes, st.k_scales, st.v_scales, st.kbar, st.state, st.seqlens)):
                assert torch.equal(x, y)
            with pytest.raises(D.DashError, match="another row"):
                pool.check()
        assert torch.equal(st.decode(q), out[k])
    pool.free([0, 1])             # row 3 now holds its pages alone
    pool.reserve(_ints(130, 0, 64, 0))
    free = _ints(130, 0, 64, 0)
    for k, st in enumerate(sts):
        st.append(V[:, :130], K[:, :130], free)
        assert torch.equal(st.decode(q)[3], out[k][3])
    pool.check()
    for st in sts:
        st.fill(K, V, [100, 0, 10, 150])   # every page has one holder: the caches start over
        assert st.seqlens.tolist() == [100, 0, 10, 150]
    pool.check()


def test_fill_of_shared_pages_in_a_graph():
    """The check runs on the device: a captured fill spares shared pages at every replay."""
    rnd = _rnd(5)
    table = torch.full((3, 8), -1, dtype=torch.int32, device="cuda")
    st = _make(3, num_pages=20, page_table=table)
    pool = D.PagePool.of([st])
    K, V, lens = rnd(3, 128, HKV, DIM), rnd(3, 128, HKV, DIM), _ints(128, 0, 0)
    pool.reserve(lens)
    st.fill(K, V, lens)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        st.fill(V, K, lens)
    graph.replay()
    swapped = st.k_codes.clone()
    st.fill(K, V, lens)
    held = st.k_codes.clone()
    assert not torch.equal(held, swapped)
    pool.fork([0], [1])
    graph.replay()
    assert torch.equal(st.k_codes, held) and st.seqlens.tolist() == [128, 128, 0]
    with pytest.raises(D.DashError, match="another row"):
        pool.check()
    pool.free([1])
    graph.replay()
    assert torch.equal(st.k_codes, swapped)
    pool.check()


def test_fill_of_a_bf16_cache_spares_shared_pages():
    rnd = _rnd(6)
    table = torch.full((3, 4), -1, dtype=torch.int32, device="cuda")
    st = D.PagedDecodeState(3, 256, HQ, HKV, 128, chunk=64, alpha=1.5, gamma=3.0, page_size=PAGE, num_pages=10, page_table=table,
                            qbar=torch.zeros(HKV, 128, device="cuda"))
    pool = D.PagePool.of([st])
    K, V = rnd(3, 150, HKV, 128), rnd(3, 150, HKV, 128)
    pool.reserve(_ints(150, 0, 60))
    st.fill(K, V, [150, 0, 60])
    st.fill(K, V, [150, 0, 60])
    pool.fork([0], [1])
    before = [t.clone() for t in (st.K, st.V, st.kbar, st.state, st.seqlens)]
    with pytest.raises(ValueError, match="another row"):
        st.fill(V, K, [150, 0, 60])
    for x, y in zip(before, (st.K, st.V, st.kbar, st.state, st.seqlens)):
        assert torch.equal(x, y)
    pool.free([1])
    st.fill(V, K, [150, 0, 60])
    assert torch.equal(st.K[int(table[0, 0])], V[0, :PAGE])


def test_rows_that_take_no_token():
    """step and graph_step with counts: rows with 0 keep their length, pages and state, an emptied row can be forked
    into, and both equal append(counts) + decode."""
    rnd = _rnd(7)
    made = []
    for _ in range(3):
        table = torch.full((4, 8), -1, dtype=torch.int32, device="cuda")
        st = _make(4, num_pages=24, page_table=table)
        made.append((st, D.PagePool.of([st])))
    K, V = rnd(4, 120, HKV, DIM), rnd(4, 120, HKV, DIM)
    for st, pool in made:
        pool.reserve(_ints(120, 60, 5, 0))
        st.fill(K, V, [120, 60, 5, 0])
        pool.free([1])
    stream = torch.cuda.Stream()
    on = [1, 0, 1, 0]
    lens = [120, 0, 5, 0]
    for t in range(75):
        if t == 40:
            for _, pool in made:
                pool.fork([0], [3])
                pool.check()
            on, lens[3] = [1, 0, 0, 1], lens[0]
        counts = _ints(*on)
        lens = [n + c for n, c in zip(lens, on)]
        ins = _step(rnd, 4)
        outs = []
        for k, (st, pool) in enumerate(made):
            pool.reserve(counts)
            if k == 0:
                st.append(ins[1], ins[2], counts)
                outs.append(st.decode(ins[0]).clone())
            elif k == 1:
                outs.append(st.graph_step(*ins, counts=counts).clone())
            else:
                stream.wait_stream(torch.cuda.current_stream())
                o = st.step(*ins, counts=counts, stream=stream)
                torch.cuda.current_stream().wait_stream(stream)
                outs.append(o.clone())
            pool.check()
            assert st.seqlens.tolist() == lens and (pool.page_table[1] == -1).all()
        assert torch.equal(outs[0], outs[1]) and torch.equal(outs[0], outs[2]) and not outs[0][1].any()
    for st, _ in made[1:]:
        _same_state(made[0][0], st)


def test_recorded_steps_with_and_without_counts():
    """One cache's recorded steps of both kinds in turn equal the eager ones; counts of another size are refused."""
    rnd = _rnd(8)
    eager, graph = _make(), _make()
    for t in range(12):
        ins, counts = _step(rnd), _ints(t % 2, 1, t % 3) if t % 4 < 2 else None
        assert torch.equal(eager.step(*ins, counts=counts).clone(), graph.graph_step(*ins, counts=counts))
    _same_state(eager, graph)
    ins, lens = _step(rnd), graph.seqlens.tolist()
    for bad in (_ints(1, 1), _ints(1, 1, 1).long(), torch.tensor([1, 1, 1], dtype=torch.int32)):
        with pytest.raises((TypeError, ValueError)):
            graph.graph_step(*ins, counts=bad)
        with pytest.raises((TypeError, ValueError)):
            graph.step(*ins, counts=bad)
    assert graph.seqlens.tolist() == lens


def test_a_step_that_is_refused_appends_nothing():
    rnd = _rnd(9)
    st = _make()
    q, k, v = _step(rnd)
    st.step(q, k, v)
    held = st.k_codes.clone()
    for bad in (q.float(), q[:2], q[:, :4], q.cpu(), q.transpose(0, 1).contiguous().transpose(0, 1), None):
        with pytest.raises((TypeError, ValueError)):
            st.step(bad, k, v)
        with pytest.raises((TypeError, ValueError)):
            st.graph_step(bad, k, v)
    off = torch.zeros(3 * HQ * DIM + 4, dtype=torch.bfloat16, device="cuda")[4:].view(3, HQ, DIM)   # 8 bytes past the alignment
    with pytest.raises(D.DashError):
        st.step(off, k, v)
    assert st.seqlens.tolist() == [1, 1, 1] and torch.equal(st.k_codes, held)


def test_a_fill_that_is_refused_changes_nothing():
    rnd = _rnd(10)
    st = _make()
    K = rnd(3, 40, HKV, DIM)
    st.fill(K, K, [40, 3, 0])
    wide = torch.zeros(3, 40, HKV, DIM + 4, dtype=torch.bfloat16, device="cuda")[..., :DIM]   # rows 136 bytes apart
    with pytest.raises(D.DashError):
        st.fill(wide, K, [40, 3, 1])
    qbar, st.qbar = st.qbar, None
    with pytest.raises(TypeError):
        st.fill(K, K, [40, 3, 1])
    st.qbar = qbar
    for bad in ([1, 2], [[1, 2, 3]]):
        with pytest.raises((TypeError, ValueError)):
            st.fill(K, K, bad)
    assert st.seqlens.tolist() == [40, 3, 0]


def test_check_sees_operations_on_other_streams():
    """check() waits for operations wherever they were enqueued, and what it clears stays apart from later ones."""
    table = torch.full((2, 4), -1, dtype=torch.int32, device="cuda")
    pool = D.PagePool(table, torch.zeros(8, dtype=torch.int32, device="cuda"), _ints(0, 0), page_size=PAGE)
    stream = torch.cuda.Stream()
    for _ in range(3):
        stream.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(stream):
            torch.cuda._sleep(20_000_000)   # some 10 ms
        pool.reserve(10000, stream=stream)
        with pytest.raises(D.DashError, match="length"):
            pool.check()
        pool.check()


def test_fork_into_a_row_that_holds_any_page():
    """A row of length 0 whose first slot is empty but a later one is not is not empty: its pages are not lost."""
    for slots, at in ((4, 2), (40, 39), (1500, 1499), (1500, 33)):
        table = torch.full((3, slots), -1, dtype=torch.int32, device="cuda")
        refs = torch.zeros(8, dtype=torch.int32, device="cuda")
        table[0, 0], table[1, at] = 5, 3
        refs[5] = refs[3] = 1
        lens = _ints(20, 0, 0)
        pool = D.PagePool(table, refs, lens, page_size=PAGE)
        before = table.clone(), refs.clone(), lens.clone()
        pool.fork([0, 0], [2, 1])
        for x, y in zip(before, (table, refs, lens)):
            assert torch.equal(x, y)
        with pytest.raises(D.DashError, match="not empty"):
            pool.check()
        pool.free([1])
        pool.fork([0, 0], [2, 1])
        pool.check()
        assert refs.tolist() == [1, 1, 0, 0, 0, 1, 0, 0] and lens.tolist() == [20, 20, 20]


def test_fork_many_rows_of_many_slots():
    """More entries than the check takes at a time, full tables beside them."""
    rows, slots = 900, 70
    table = torch.full((rows, slots), -1, dtype=torch.int32, device="cuda")
    refs = torch.zeros(200, dtype=torch.int32, device="cuda")
    table[:2] = torch.arange(2 * slots, dtype=torch.int32, device="cuda").view(2, slots)
    refs[: 2 * slots] = 1
    lens = torch.zeros(rows, dtype=torch.int32, device="cuda")
    lens[:2] = slots * PAGE
    pool = D.PagePool(table, refs, lens, page_size=PAGE)
    src = torch.arange(rows - 2, device="cuda").int() % 2
    dst = torch.arange(2, rows, device="cuda").int()
    table[700, 69] = 150
    refs[150] = 1
    before = table.clone(), refs.clone()
    pool.fork(src, dst)
    with pytest.raises(D.DashError, match="not empty"):
        pool.check()
    assert torch.equal(before[0], table) and torch.equal(before[1], refs)
    pool.free([700])
    pool.fork(src, dst)
    pool.check()
    assert torch.equal(table[2:], table[:2][src.long()]) and refs[: 2 * slots].tolist() == [450] * (2 * slots)


def test_reserve_looks_from_the_next_token_on():
    """Slots before the one of the next token are left as they are: what a row without a page there dropped reads as
    zeros, not as what a page held before."""
    rnd = _rnd(11)
    table = torch.full((2, 8), -1, dtype=torch.int32, device="cuda")
    st = _make(2, num_pages=12, page_table=table)
    pool = D.PagePool.of([st])
    for t in (st.k_codes, st.v_codes, st.k_scales, st.v_scales):
        t.fill_(0x31)   # what other rows left there
    K = rnd(2, 2 * PAGE, HKV, DIM)
    pool.reserve(_ints(PAGE, PAGE))
    st.append(K, K, _ints(2 * PAGE, PAGE))   # row 0 has no page for its second half
    pool.reserve(_ints(5, 5))
    pool.check()
    assert (table[0] >= 0).tolist() == [True, False, True] + [False] * 5 and (table[1, :2] >= 0).all()
    assert not st.load(PAGE, PAGE)[0][0].any()
