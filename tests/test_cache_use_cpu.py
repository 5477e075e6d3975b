"""Refusals of the cache classes that need no GPU: nothing is launched."""
import os
import re

import pytest
import torch

import adaptive_sparse_hierarchical_b200 as D
from adaptive_sparse_hierarchical_b200.build import build


@pytest.fixture(scope="module", autouse=True)
def _built():
    build()


def _q4(**kw):
    return D.Q4DecodeState(4, 512, 8, 2, 64, **{**dict(chunk=32, alpha=1.5, gamma=2.0, page_size=64, num_pages=40, device="cpu"), **kw})


BAD_TABLES = [torch.zeros(3, 8, dtype=torch.int32), torch.zeros(1, 32, dtype=torch.int32), torch.zeros(0, 8, dtype=torch.int32),
              torch.zeros(32, dtype=torch.int32), torch.zeros(4, 8, 1, dtype=torch.int32)]


@pytest.mark.parametrize("table", BAD_TABLES, ids=[str(tuple(t.shape)) for t in BAD_TABLES])
def test_page_tables_of_other_shapes(table):
    """A table with fewer rows than sequences would be read, and its entries followed, beyond its end."""
    with pytest.raises(ValueError, match="page_table"):
        _q4(page_table=table)
    assert _q4(page_table=torch.zeros(4, 9, dtype=torch.int32)).kv.max_pages == 9
    assert _q4(page_table=torch.zeros(6, 8, dtype=torch.int32)).page_table.shape == (6, 8)   # (further rows are not read)
    assert _q4().page_table.shape == (4, 8)


@pytest.mark.parametrize("table", BAD_TABLES, ids=[str(tuple(t.shape)) for t in BAD_TABLES])
def test_page_tables_of_other_shapes_bf16(table):
    def make(t):
        return D.PagedDecodeState(4, 512, 8, 2, 128, chunk=64, alpha=1.5, gamma=2.0, page_size=64, num_pages=40, page_table=t,
                                  device="cpu")

    with pytest.raises(ValueError, match="page_table"):
        make(table)
    for rows in (4, 6):
        assert make(torch.zeros(rows, 9, dtype=torch.int32)).pk.max_pages == 9


def test_token_numbers_beyond_32_bits():
    """The rows of load are numbered in 32 bits with the last block's spare ones, and a C int holds the number."""
    lib, i = D.load(), 256
    p = D.params(batch=1, seqlen=512, h_q=4, h_kv=2, d_h=64, chunk=32, alpha=1.5, gamma=2.0, k_strides=(1 << 40, 128, 64),
                 v_strides=(1 << 40, 128, 64))
    pool = torch.zeros(8, 2, 64, 32, dtype=torch.uint8)
    kv = D.q4_kv(pool, pool[..., :2].contiguous(), pool, pool[..., :2].contiguous(), torch.zeros(1, 8, dtype=torch.int32), page_size=64)
    for n in ((1 << 31) - 1, (1 << 30) + 1):
        assert lib.dash_load_q4(p, kv, None, 0, n, i, i, i, None) == -2   # DASH_EUNSUPPORTED
    st = _q4(qbar=torch.zeros(2, 64))
    many = torch.zeros(64, dtype=torch.bfloat16).expand(4, (1 << 32) + 1, 2, 64)
    for call in (lambda: st._check("append", many, many, None, "counts"), lambda: st._check("load", many, many, None, "start")):
        with pytest.raises(ValueError, match="32 bits"):
            call()


def test_no_read_only_loads_of_what_a_running_kernel_may_write():
    """The cache's kernels start before the one ahead of them ends (programmatic dependent launch).  What that one writes
    (tables, lengths, summaries, logits) may then not be read by the read-only path, which holds only for memory
    that nobody writes while the kernel runs: neither __ldg nor const __restrict__ pointers."""
    src = os.path.join(os.path.dirname(D.__file__), "csrc")
    for name in ("q4.cuh", "q4_cache.cu", "q4_decode.cu", "q4_route.cuh", "q4_route.cu", "pages.cuh", "pages.cu"):
        text = open(os.path.join(src, name)).read()
        text = re.sub(r"//[^\n]*", "", text)
        # (the page table, where the routing's launches lie between the kernel and whoever wrote it)
        text = text.replace("!SOLO && !a.dense ? __ldg(e) : table_entry(e)", "", 1)
        assert not re.findall(r"__ldg|__restrict__|ld\.global\.nc", text), name


@pytest.mark.parametrize("name", ["k_scales", "v_codes", "kbar", "state"])
def test_a_cache_that_is_refused_is_not_registered_in_part(name):
    """add of a cache one of whose tensors is refused registers none of them; put right, it is registered once."""
    table = torch.full((4, 8), -1, dtype=torch.int32)
    st, other = _q4(page_table=table), _q4(page_table=table)
    pool = D.PagePool.of([st])
    arrays, rows = pool.pg.num_arrays, pool.pg.num_rows
    right = getattr(other, name)
    setattr(other, name, right.repeat_interleave(2, -1)[..., ::2])   # the same values, not contiguous
    with pytest.raises(ValueError):
        pool.add(other)
    assert (pool.pg.num_arrays, pool.pg.num_rows) == (arrays, rows)
    setattr(other, name, right)
    seqlens, other.seqlens = other.seqlens, None   # not a tensor at all
    with pytest.raises(AttributeError):
        pool.add(other)
    assert (pool.pg.num_arrays, pool.pg.num_rows) == (arrays, rows)
    other.seqlens = seqlens
    pool.add(other)
    assert (pool.pg.num_arrays, pool.pg.num_rows) == (2 * arrays, 2 * rows + 1)
