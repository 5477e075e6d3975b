"""Page operations on the GPU (dash_pages_*) against a plain model on the host, and runs of them under the
caches that use them."""
import random

import numpy as np
import pytest
import torch

import adaptive_sparse_hierarchical_b200 as D

pytestmark = pytest.mark.gpu

PAGE = 64


class Model:
    """The definition, on the host: tables, counts, lengths and the contents of one int64 per page."""

    def __init__(self, batch, slots, pages):
        self.table = -np.ones((batch, slots), np.int64)
        self.refs = np.zeros(pages, np.int64)
        self.lens = np.zeros(batch, np.int64)
        self.data = np.arange(pages) * 1000

    def free_pages(self, n):
        at = np.flatnonzero(self.refs == 0)[:n]
        return at if len(at) == n else None

    def reserve(self, add):
        want = [(b, s) for b, a in enumerate(add) if a > 0
                for s in range(self.lens[b] // PAGE, -(-(self.lens[b] + a) // PAGE)) if self.table[b, s] < 0]
        pages = self.free_pages(len(want))
        if pages is None:
            return 4
        for (b, s), p in zip(want, pages):
            self.table[b, s] = p
            self.refs[p] = 1

    def fork(self, src, dst):
        part = [i for i, s in enumerate(src) if self.lens[s] % PAGE]
        pages = self.free_pages(len(part))
        if pages is None:
            return 4
        own = dict(zip(part, pages))
        for i, (s, d) in enumerate(zip(src, dst)):
            full = self.lens[s] // PAGE
            self.table[d] = -1
            self.table[d, :full] = self.table[s, :full]
            for p in self.table[s, :full]:
                self.refs[p] += 1
            if i in own:
                self.table[d, full] = own[i]
                self.refs[own[i]] = 1
                self.data[own[i]] = self.data[self.table[s, full]]
            self.lens[d] = self.lens[s]

    def free(self, rows):
        for b in set(rows):
            for p in self.table[b]:
                if p >= 0:
                    self.refs[p] -= 1
            self.table[b] = -1
            self.lens[b] = 0

    def compact(self):
        U = int((self.refs > 0).sum())
        holes, movers = np.flatnonzero(self.refs[:U] == 0), np.flatnonzero(self.refs[U:] > 0) + U
        to = np.arange(len(self.refs))
        to[movers] = holes
        self.data[holes] = self.data[movers]
        self.refs[holes], self.refs[movers] = self.refs[movers], 0
        self.table = np.where(self.table >= 0, to[self.table], -1)
        return U


def _pool(m, device="cuda"):
    """A PagePool over the model's state, two pools of different page sizes that carry its data, and row arrays."""
    ints = lambda x: torch.tensor(x, dtype=torch.int32, device=device)   # noqa: E731
    pool = D.PagePool(ints(m.table), ints(m.refs), ints(m.lens), page_size=PAGE)
    n = len(m.refs)
    a = torch.tensor(m.data, device=device)[:, None].repeat(1, 1100)                        # 8800 bytes: two pieces
    wide = torch.tensor(m.data, device=device)[:, None].repeat(1, 16)
    b = wide[:, :6]                                                                         # 48 of 128 bytes
    a[:, 1] = torch.arange(n, device=device)
    a[:, 1] = a[:, 0]
    pool.add_pages(a)
    pool.add_pages(b)
    batch, slots = m.table.shape
    kbar = torch.zeros(batch, 3, slots * PAGE // 32, 8, device=device)
    state = torch.zeros(batch, 3, 5, device=device)                                         # rows of 60 bytes
    extra = ints(m.lens.copy())
    pool.add_rows(kbar, unit_tokens=32)
    pool.add_rows(state)
    pool.add_rows(extra, clear=True)
    return pool, a, wide, kbar, state, extra


def _same(pool, m, a, wide):
    assert np.array_equal(pool.page_table.cpu().numpy(), m.table)
    assert np.array_equal(pool.refs.cpu().numpy(), m.refs)
    assert np.array_equal(pool.seqlens.cpu().numpy(), m.lens)
    got = a.cpu().numpy()
    assert np.array_equal(got, np.repeat(m.data[:, None], 1100, 1))
    w = wide.cpu().numpy()
    assert np.array_equal(w[:, :6], np.repeat(m.data[:, None], 6, 1))
    assert np.array_equal(w[:, 6:], np.repeat((np.arange(len(w)) * 1000)[:, None], 10, 1))   # between pages: untouched


@pytest.mark.parametrize("seed,batch,slots,pages", [(0, 6, 5, 40), (1, 40, 3, 50), (2, 3, 1500, 3500), (3, 5, 4, 9000),
                                                    (4, 1, 1, 1)])
def test_random_runs(seed, batch, slots, pages):
    """Random reserve / grow / fork / free / compact / copy, checked after each, refusals included."""
    rng = random.Random(seed)
    m = Model(batch, slots, pages)
    if seed == 3:   # pages beyond one step of the scans are in use
        m.refs[:8500] = 1
        m.refs[17] = m.refs[8300] = 0
    pool, a, wide, kbar, state, extra = _pool(m)
    refused = 0
    for step in range(60):
        op = rng.choice(["reserve", "reserve", "fork", "fork", "free", "compact", "copy"])
        code = None
        if op == "reserve":
            add = [rng.choice([0, 0, 1, PAGE // 2, PAGE, rng.randrange(0, slots * PAGE)]) for _ in range(batch)]
            add = [min(x, slots * PAGE - int(n)) for x, n in zip(add, m.lens)]
            code = m.reserve(add)
            pool.reserve(torch.tensor(add, dtype=torch.int32, device="cuda"))
            if code is None:   # the caches write tokens there and move the lengths
                m.lens += np.maximum(add, 0)
                pool.seqlens.copy_(torch.tensor(m.lens, dtype=torch.int32))
                extra.copy_(pool.seqlens)
                kbar.random_(0, 1000)
                state.random_(0, 1000)
        elif op == "fork":
            empty = [b for b in range(batch) if m.lens[b] == 0 and m.table[b, 0] < 0]
            dst = rng.sample(empty, rng.randrange(0, len(empty) + 1))
            others = [b for b in range(batch) if b not in dst]
            if not others:
                continue
            src = [rng.choice(others) for _ in dst]
            before = kbar.clone(), state.clone(), extra.clone()
            code = m.fork(src, dst)
            pool.fork(src, dst)
            if code is None:
                for s, d in zip(src, dst):
                    n = int(m.lens[s]) // 32
                    before[0][d, :, :n] = before[0][s, :, :n]
                    before[1][d], before[2][d] = before[1][s], before[2][s]
            for x, y in zip(before, (kbar, state, extra)):
                assert torch.equal(x, y)
        elif op == "free":
            rows = [rng.randrange(batch) for _ in range(rng.randrange(0, 1 + batch // 2))]
            m.free(rows)
            pool.free(rows)
            assert not extra[rows].any()
        elif op == "compact":
            U = m.compact()
            assert pool.compact().item() == U
        else:
            at = rng.sample(range(pages), pages)
            n = rng.randrange(0, pages // 2 + 1)
            src = [rng.choice(at[n:]) for _ in range(n)] if n < pages else []
            m.data[at[:n]] = m.data[src]
            pool.copy(src, at[:n])
        _same(pool, m, a, wide)
        assert int(pool.status.item()) == (code or 0), op
        if code:
            refused += 1
            with pytest.raises(D.DashError):
                pool.check()
        pool.check()
    if seed in (1, 2):   # fewer pages than the rows can hold
        assert refused


def test_copy_onto_itself_and_shared_source():
    m = Model(1, 1, 8)
    pool, a, wide, *_ = _pool(m)
    pool.copy([3, 3, 5], [0, 1, 5])   # 5 onto itself, 3 twice
    m.data[[0, 1]] = m.data[3]
    _same(pool, m, a, wide)
    pool.copy([5, 5], [5, 2])         # 5 is "written" with its own contents and read
    m.data[2] = m.data[5]
    _same(pool, m, a, wide)
    pool.check()


@pytest.mark.parametrize("what,code", [
    (lambda p: p.copy([0, 8], [1, 2]), 1), (lambda p: p.copy([0, 1], [-1, 2]), 1), (lambda p: p.copy([0, 1], [2, 2]), 2),
    (lambda p: p.copy([0, 1], [1, 2]), 2), (lambda p: p.fork([0, 0], [2, 2]), 2), (lambda p: p.fork([0], [1]), 3),
    (lambda p: p.fork([0], [5]), 1), (lambda p: p.fork([-1], [2]), 1), (lambda p: p.fork([0, 2], [2, 3]), 2),
    (lambda p: p.fork([4], [3]), 1), (lambda p: p.reserve(10000), 5), (lambda p: p.reserve(PAGE * 3), 4),
])
def test_refusals_change_nothing(what, code):
    """Requests that cannot be met: nothing moves, status tells why, check() raises and clears it."""
    m = Model(5, 6, 8)
    m.table[0, :2] = [4, 2]
    m.lens[0] = 100
    m.table[1, :2] = [4, 6]
    m.lens[1] = 90
    m.refs[[4, 2, 6]] = [2, 1, 1]
    m.lens[4] = 10    # a row whose page is missing
    pool, a, wide, kbar, state, extra = _pool(m)
    what(pool)
    _same(pool, m, a, wide)
    assert pool.status.item() == code
    assert extra.tolist() == m.lens.tolist()
    with pytest.raises(D.DashError):
        pool.check()
    pool.check()


def test_free_reports_bad_rows_and_frees_the_others():
    m = Model(3, 2, 6)
    m.reserve([70, 10, 0])
    m.lens[:] = [70, 10, 0]
    pool, a, wide, *_ = _pool(m)
    pool.free([7, 0, -1, 0, 2])
    m.free([0])
    _same(pool, m, a, wide)
    assert pool.status.item() == 1


def test_many_arrays():
    """More arrays than one mover launch takes."""
    m = Model(4, 3, 12)
    m.reserve([100, 64, 0, 0])
    m.lens[:] = [100, 64, 0, 0]
    pool, a, wide, *_ = _pool(m)
    more = [torch.full((12, 2 + 2 * (i % 5)), i, dtype=torch.int64, device="cuda") + torch.arange(12, device="cuda")[:, None] * 100
            for i in range(150)]
    rows = [torch.full((4, 3), 10 * i, dtype=torch.int32, device="cuda") + torch.arange(4, dtype=torch.int32, device="cuda")[:, None]
            for i in range(130)]
    for t in more:
        pool.add_pages(t)
    for i, t in enumerate(rows):
        pool.add_rows(t, clear=i % 2 == 1)
    pool.fork([0, 1], [2, 3])
    m.fork([0, 1], [2, 3])
    _same(pool, m, a, wide)
    new = int(m.table[2, 1])
    for i, t in enumerate(more):
        want = i + torch.arange(12) * 100
        want[new] = i + 100 * m.table[0, 1]
        assert torch.equal(t[:, 0].cpu(), want) and torch.equal(t[:, -1].cpu(), want)
    for i, t in enumerate(rows):
        assert t[:, 2].tolist() == [10 * i, 10 * i + 1, 10 * i, 10 * i + 1]
    pool.free([1])
    m.free([1])
    for i, t in enumerate(rows):
        assert t[1].tolist() == ([0] * 3 if i % 2 else [10 * i + 1] * 3)
    pool.free([0, 2])
    m.free([0, 2])
    pool.compact()
    m.compact()
    _same(pool, m, a, wide)
    for i, t in enumerate(more):   # row 3's page moved to the front
        assert m.table[3, 0] == 0 and t[0, 0].item() == i + 100 * 2


def _serve(kind, layers, graph):
    """Prefill, fork, decode, free, compact, decode: rows over shared pages give what a private cache gives."""
    b, cap, hq, hkv, d, B = 6, 512, 8, 2, 128, 64
    slots, pages = cap // PAGE, 40
    table = torch.full((b, slots), -1, dtype=torch.int32, device="cuda")
    g = torch.Generator(device="cuda").manual_seed(5)
    rnd = lambda *s: torch.randn(*s, device="cuda", generator=g).bfloat16()   # noqa: E731
    qbar = torch.randn(hkv, d, device="cuda", generator=g) * 0.2
    kw = dict(chunk=B, alpha=1.5, gamma=3.0, page_size=PAGE, qbar=qbar)
    if kind == "q4":
        shared = [D.Q4DecodeState(b, cap, hq, hkv, d, num_pages=pages, page_table=table, **kw) for _ in range(layers)]
        alone = [D.Q4DecodeState(b, cap, hq, hkv, d, **kw) for _ in range(layers)]
    else:
        shared = [D.PagedDecodeState(b, cap, hq, hkv, d, num_pages=pages, page_table=table, **kw) for _ in range(layers)]
        alone = [D.PagedDecodeState(b, cap, hq, hkv, d, num_pages=b * slots,
                                    page_table=torch.arange(b * slots).view(b, slots), **kw) for _ in range(layers)]
        for s in shared + alone:
            s.state[..., d] = -torch.inf
    pool = D.PagePool.of(shared)
    toks = [(rnd(b, cap, hkv, d), rnd(b, cap, hkv, d)) for _ in range(layers)]
    lens = [200, 64, 0, 0, 0, 0]
    pool.reserve(torch.tensor(lens, dtype=torch.int32, device="cuda"))
    for s, (K, V) in zip(shared, toks):
        if kind == "q4":
            s.fill(K, V, lens)
        else:
            s.fill(K[:, :200].contiguous(), V[:, :200].contiguous(), lens)
    src, dst = [0, 0, 1], [2, 4, 5]
    pool.fork(src, dst)
    lens = [200, 64, 200, 0, 200, 64]
    rows = [0, 1, 0, 3, 0, 1]
    for s, (K, V) in zip(alone, toks):
        K, V = K[rows], V[rows]
        s.fill(K, V, lens) if kind == "q4" else s.fill(K[:, :200].contiguous(), V[:, :200].contiguous(), lens)
    live = [i for i, n in enumerate(lens) if n]

    def steps(n):
        outs = []
        for _ in range(n):
            pool.reserve(1)
            for s, t in zip(shared, alone):
                q, k, v = rnd(b, hq, d), rnd(b, hkv, d), rnd(b, hkv, d)
                o, p = s.step(q, k, v), t.step(q, k, v)
                outs.append(torch.equal(o[live], p[live]))
        return all(outs)

    assert steps(70)
    pool.check()
    pool.free([0, 3])
    live.remove(0)
    used = int(pool.compact().item())
    assert used == int((pool.refs > 0).sum()) and int(pool.page_table.max()) < used
    for t in alone:
        t.seqlens[[0, 3]] = 0
        if kind == "q4":
            continue
        t.state[[0, 3]] = 0
        t.state[[0, 3], :, d] = -torch.inf
    for s in shared:   # the freed rows are empty in every layer
        assert not s.seqlens[[0, 3]].any() and (s.state[[0, 3], :, d] == -torch.inf).all() and not s.state[[0, 3], :, :d].any()
    live = [0, 1, 2, 3, 4, 5]
    assert steps(70)   # the emptied rows start over, past a chunk's end
    for s, t in zip(shared, alone):
        for i, n in enumerate(s.seqlens.tolist()):
            assert torch.equal(s.kbar[i, :, : n // B], t.kbar[i, :, : n // B]) and torch.equal(s.state[i], t.state[i])
    pool.check()


@pytest.mark.parametrize("kind,layers", [("q4", 1), ("q4", 3), ("bf16", 2)])
def test_serving_over_shared_pages(kind, layers):
    _serve(kind, layers, False)


def test_captured_run():
    """free + fork + reserve captured into one graph and replayed equals the eager calls."""
    m = Model(6, 4, 40)
    m.reserve([150, 70, 0, 0, 0, 0])
    m.lens[:] = [150, 70, 0, 0, 0, 0]
    pool, a, wide, *_ = _pool(m)
    src = torch.tensor([0, 1, 0], dtype=torch.int32, device="cuda")
    dst = torch.tensor([2, 3, 5], dtype=torch.int32, device="cuda")
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        pool.free(dst)
        pool.fork(src, dst)
        pool.reserve(30)
    for s in ([0, 1, 0], [1, 1, 1], [0, 0, 1]):
        src.copy_(torch.tensor(s))
        graph.replay()
        m.free([2, 3, 5])
        assert m.fork(s, [2, 3, 5]) is None and m.reserve([30] * 6) is None
        _same(pool, m, a, wide)
    pool.check()


def test_fork_in_a_large_batch():
    """More rows than a plan's shared memory marks, all 1024 entries of a call, and the marks' checks there."""
    m = Model(5000, 2, 3000)
    m.reserve([100 if b < 40 else 0 for b in range(5000)])
    m.lens[:40] = 100
    pool, a, wide, *_ = _pool(m)
    src, dst = [i % 40 for i in range(1024)], list(range(4999, 4999 - 1024, -1))
    pool.fork(src, dst)
    m.fork(src, dst)
    _same(pool, m, a, wide)
    pool.check()
    pool.fork([0, 1, 2], [50, 60, 50])
    _same(pool, m, a, wide)
    with pytest.raises(D.DashError, match="twice"):
        pool.check()


def test_rows_of_odd_units():
    """Row arrays whose runs are copied word by word, several heads, ragged lengths."""
    m = Model(4, 3, 12)
    m.reserve([100, 30, 0, 0])
    m.lens[:] = [100, 30, 0, 0]
    pool, a, wide, *_ = _pool(m)
    t = torch.randint(0, 1000, (4, 3, 6, 3), dtype=torch.int32, device="cuda")
    pool.add_rows(t, unit_tokens=32)
    want = t.clone()
    pool.fork([0, 1], [3, 2])
    m.fork([0, 1], [3, 2])
    want[3, :, :3] = want[0, :, :3]
    assert torch.equal(t, want)
    _same(pool, m, a, wide)


def test_refused_registrations():
    m = Model(3, 2, 6)
    pool, *_ = _pool(m)
    for bad in (torch.zeros(5, 4, device="cuda"), torch.zeros(6, 4), torch.zeros(6, 3, device="cuda"),
                torch.zeros(6, 4, 4, device="cuda").transpose(1, 2), torch.zeros(1, 4, device="cuda").expand(6, 4)):
        with pytest.raises(ValueError):
            pool.add_pages(bad)
    for bad in (torch.zeros(2, 4, device="cuda"), torch.zeros(3, 4, 4, device="cuda").transpose(1, 2),
                torch.zeros(1, 4, device="cuda").expand(3, 4), torch.zeros(3, 3, dtype=torch.int16, device="cuda")):
        with pytest.raises(ValueError):
            pool.add_rows(bad)
    with pytest.raises(TypeError):
        pool.free(torch.tensor([1], device="cuda"))
    with pytest.raises(ValueError):
        pool.fork([0, 1], [2])
    with pytest.raises(ValueError):
        pool.reserve((1 << 32) + 1)
    pool.free([0])
    pool.check()


def test_lists_on_another_stream():
    """Calls on a stream of their own take their lists there too."""
    m = Model(4, 3, 12)
    m.reserve([100, 64, 0, 0])
    m.lens[:] = [100, 64, 0, 0]
    pool, a, wide, *_ = _pool(m)
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    pool.fork([0, 1], [2, 3], stream=stream)
    pool.reserve(50, stream=stream)
    pool.free([0], stream=stream.cuda_stream)
    pool.compact(stream=stream)
    torch.cuda.current_stream().wait_stream(stream)
    m.fork([0, 1], [2, 3])
    m.reserve([50] * 4)
    m.free([0])
    m.compact()
    _same(pool, m, a, wide)
