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
