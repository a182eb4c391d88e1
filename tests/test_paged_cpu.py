"""Host-side checks of the one-kind paged caches' entry points and of their Python helpers, without a GPU."""

import ctypes

import pytest
import torch

from int2_rotated_kv_oscar_gb300 import abi, build
from int2_rotated_kv_oscar_gb300 import cache as kv


@pytest.fixture(scope="module")
def lib():
    build.build()
    return abi.load(build_if_missing=False)


def test_null_arguments_are_refused(lib):
    assert lib.oscar_rope_table(None, None, 1, 128, 1e6, None) == 1
    assert lib.oscar_rope_append_bf16(None, None, None, None) == 1
    assert lib.oscar_rope_append_int4(None, None, None, None) == 1
    assert lib.oscar_int4_to_bf16(None, None, None, None, None, 1, None) == 1
    assert lib.oscar_window_attention_bf16(None, None, None, None, 0, None) == 1
    assert lib.oscar_window_attention_int4(None, None, None, None, 0, None) == 1
    assert lib.oscar_window_workspace_bytes(None) == 0


def test_struct_layouts_match_the_header():
    assert abi.INT4_BLOCK_BYTES == 8704
    view, app, win = abi.oscar_int4_cache_view, abi.oscar_rope_append_args, abi.oscar_window_args
    assert (view.page_table.offset, view.batch.offset, ctypes.sizeof(view)) == (16, 28, 32)
    assert (app.rope.offset, app.interleaved.offset, app.pos.offset, app.n_tokens.offset, ctypes.sizeof(app)) == (
        64, 80, 88, 104, 112)
    assert (win.q_stride.offset, win.n_tokens.offset, win.sm_scale.offset, ctypes.sizeof(win)) == (40, 48, 68, 72)


def test_helpers_refuse_what_the_structs_cannot_say():
    q = torch.zeros(3, 4, 128, dtype=torch.bfloat16)
    i = torch.zeros(3, dtype=torch.int32)
    assert kv.window_args(q, torch.zeros_like(q), i, i, 10).q_stride == 512
    assert kv.window_args(torch.zeros(3, 6, 128, dtype=torch.bfloat16)[:, 1:5], torch.zeros_like(q), i, i, 10).q_stride == 768
    with pytest.raises(ValueError):  # heads that do not lie side by side
        kv.window_args(torch.zeros(3, 4, 130, dtype=torch.bfloat16)[:, :, :128], torch.zeros_like(q), i, i, 10)
    with pytest.raises(ValueError):  # a result with gaps
        kv.window_args(q, torch.zeros(3, 6, 128, dtype=torch.bfloat16)[:, 1:5], i, i, 10)
    for bad in (q.float(), q[:2], q[:, :2]):  # another type, fewer rows, fewer heads than q
        with pytest.raises(ValueError):
            kv.window_args(q, bad.contiguous(), i, i, 10)
    with pytest.raises(ValueError):
        kv.window_args(q, torch.zeros_like(q), i.long(), i, 10)
    with pytest.raises(ValueError):
        kv.window_args(q, torch.zeros_like(q), torch.zeros(6, dtype=torch.int32)[::2], i, 10)
    k = torch.zeros(3, 2, 128, dtype=torch.bfloat16)
    rope = torch.zeros(16, 128)
    assert kv.rope_append_args(k, k.clone(), i, q=q, q_out=q, rope=rope).rotary_dim == 128
    for change in (dict(v=k[:2]), dict(q=q), dict(q=q[:2], q_out=q[:2]), dict(q=q, q_out=q[:, :2]), dict(rope=rope.double()),
                   dict(rope=rope[:, ::2]), dict(rope=rope[0]), dict(pos=i.long()), dict(cu_seqlens=i.long())):
        a = dict(k=k, v=k.clone(), pos=i)
        a.update(change)
        with pytest.raises(ValueError):
            kv.rope_append_args(**a)
    table = torch.zeros(2, 4, dtype=torch.int32)
    pool = torch.zeros(3, 2, 64, 128, dtype=torch.bfloat16)
    codes = torch.zeros(3, 2, abi.INT4_BLOCK_BYTES, dtype=torch.uint8)
    assert (kv.bf16_view(pool, pool.clone(), table).batch, kv.int4_view(codes, table).max_pages_per_req) == (2, 4)
    for bad in ((pool, pool[:2], table), (pool.half(), pool.half(), table), (pool, pool, table.long()), (pool, pool, table[0])):
        with pytest.raises(ValueError):
            kv.bf16_view(*bad)
    for bad in ((codes[:, :, :8192].contiguous(), table), (codes.char(), table), (codes, table.long()), (codes, table[:, ::2])):
        with pytest.raises(ValueError):
            kv.int4_view(*bad)
