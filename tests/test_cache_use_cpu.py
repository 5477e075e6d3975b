"""Refusals of the cache classes that need no GPU: nothing is launched."""
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
