"""The paged caches' Python helpers refuse tensors that the kernels would read or write past their ends, without a GPU."""

import pytest
import torch

from int2_rotated_kv_oscar_gb300 import abi, build
from int2_rotated_kv_oscar_gb300 import cache as kv


@pytest.fixture(scope="module", autouse=True)
def lib():
    build.build()


def ints(n):
    return torch.zeros(n, dtype=torch.int32)


def test_positions_and_lengths_of_every_request():
    q = torch.zeros(3, 4, 128, dtype=torch.bfloat16)
    k = torch.zeros(3, 2, 128, dtype=torch.bfloat16)
    assert kv.window_args(q, q.clone(), ints(3), ints(4), 10).n_tokens == 3
    assert kv.window_args(q, q.clone(), ints(1), ints(1), 10, cu_seqlens=ints(2)).n_tokens == 3
    for pos, lens, cu in ((2, 3, None), (3, 2, None), (2, 3, 4), (3, 2, 4), (3, 3, 0)):
        with pytest.raises(ValueError):
            kv.window_args(q, q.clone(), ints(pos), ints(lens), 10, cu_seqlens=None if cu is None else ints(cu))
    with pytest.raises(ValueError):
        kv.window_args(q, q.clone(), torch.zeros(3, 1, dtype=torch.int32), ints(3), 10)
    assert kv.rope_append_args(k, k.clone(), ints(3)).n_tokens == 3
    assert kv.rope_append_args(k, k.clone(), ints(1), cu_seqlens=ints(2)).n_tokens == 3
    for pos, cu in ((2, None), (2, 4), (3, 0)):
        with pytest.raises(ValueError):
            kv.rope_append_args(k, k.clone(), ints(pos), cu_seqlens=None if cu is None else ints(cu))


def test_read_back_and_table_check_their_tensors():
    pages = torch.zeros(3, 2, abi.INT4_BLOCK_BYTES, dtype=torch.uint8)
    pool = torch.zeros(3, 2, 64, 128, dtype=torch.bfloat16)
    table = torch.zeros(2, 3, dtype=torch.int32)
    views = kv.int4_view(pages, table), kv.bf16_view(pool, pool.clone(), table)

    def read(pos, count):
        abi.oscar_int4_to_bf16(None, *views, pos, count, 4)

    for pos, count in ((ints(2).long(), ints(2)), (ints(2), ints(2).long()), (ints(1), ints(2)), (ints(2), ints(1)),
                       (ints(4)[::2], ints(2)), (ints(2), ints(4)[::2])):
        with pytest.raises(ValueError):
            read(pos, count)
    with pytest.raises(abi.OscarError):  # these tensors are right: the library refuses the missing context
        read(ints(2), ints(3))
    with pytest.raises(abi.OscarError):  # addresses are taken as they are
        read(ints(2).data_ptr(), ints(2).data_ptr())
    for bad in (torch.zeros(8, 128, dtype=torch.bfloat16), torch.zeros(8, 256)[:, ::2], torch.zeros(1024),
                torch.zeros(8, 128, dtype=torch.float64)):
        with pytest.raises(ValueError):
            abi.oscar_rope_table(None, bad, 1e6)
    with pytest.raises(abi.OscarError):
        abi.oscar_rope_table(None, torch.zeros(8, 128), 1e6)


def test_the_4_bit_cache_as_a_class():
    c = kv.Int4PagedCache(2, 5, 3, 4, device="cpu")
    v = c.view()
    assert (v.num_pages, v.max_pages_per_req, v.batch) == (5, 4, 3)
    assert (v.pages, v.page_table) == (c.pages.data_ptr(), c.page_table.data_ptr())
    assert not c.pages.any() and c.pages.shape == (5, 2, abi.INT4_BLOCK_BYTES)


def test_rows_that_share_memory():
    """One row broadcast to all tokens has a stride of 0, which the structs take for packed rows."""
    q = torch.zeros(3, 4, 128, dtype=torch.bfloat16)
    k = torch.zeros(3, 2, 128, dtype=torch.bfloat16)
    assert kv.window_args(q[:1].expand(1, 4, 128), q[:1].clone(), ints(1), ints(1), 10).q_stride == 512
    with pytest.raises(ValueError):
        kv.window_args(q[:1].expand(3, 4, 128), q.clone(), ints(3), ints(3), 10)
    rows = torch.zeros(3 * 256 + 256, dtype=torch.bfloat16)
    for bad in (k[:1].expand(3, 2, 128), rows.as_strided((3, 2, 128), (128, 128, 1))):
        for change in (dict(k=bad), dict(v=bad), dict(q=bad, q_out=k.clone()), dict(q=k.clone(), q_out=bad)):
            a = dict(k=k, v=k.clone(), pos=ints(3))
            a.update(change)
            with pytest.raises(ValueError):
                kv.rope_append_args(**a)
