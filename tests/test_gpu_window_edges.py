"""Calls of the windowed attention at its launch rules' edges: many rows, wrong host bounds, shared contexts."""

import numpy as np
import pytest
import torch

from int2_rotated_kv_oscar_gb300 import abi
from int2_rotated_kv_oscar_gb300 import cache as kv
from paged_harness import DEV, context, f64
from test_gpu_window import Case, steps

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("int4", [False, True])
@pytest.mark.parametrize("lengths", [range(1, 34), range(5, 125, 3), [64 * i for i in range(1, 9)]])
def test_many_single_tokens(lengths, int4):
    """Past 32 rows a block adds the lengths up in shared memory; from 32 pairs on the 4-bit blocks are the smaller ones."""
    c = Case(7, 1, steps(*lengths), 70, 3, int4, seed=300)
    c.check()
    c.close()


def test_more_rows_than_a_block_adds_up():
    """Past 1024 rows a block of the 4-bit attention takes a whole pair."""
    c = Case(2, 1, [(0, 1030, 1030), (20, 3, 15), (60, 4, 64)], 30, 1, True, seed=301)
    c.check()
    c.close()


@pytest.mark.parametrize("Hq, Hkv", [(7, 1), (8, 1), (12, 2), (10, 2), (4, 4)])
@pytest.mark.parametrize("spans", [[(0, 2, 2), (700, 40, 740)], [(1500, 17, 1517)]])
def test_chunks_of_every_head_ratio(Hq, Hkv, spans):
    c = Case(Hq, Hkv, spans, 600, 5, False, seed=302)
    c.check()
    c.close()


@pytest.mark.parametrize("int4", [False, True])
@pytest.mark.parametrize("spans", [steps(900, 64, 1500), [(2000, 40, 2040), (0, 150, 150)]])
def test_wrong_host_bound_of_the_lengths(spans, int4):
    """max_ctx_len below the lengths on the device, and far above them."""
    c = Case(8, 2, spans, -1, 0, int4, seed=303)
    for bound in (0, 1, 100, 1 << 20, 2 ** 31 - 1):
        a = c.args()
        a.max_ctx_len = bound
        c.out.fill_(9.0)
        fn = abi.oscar_window_attention_int4 if int4 else abi.oscar_window_attention_bf16
        fn(c.ctx, c.view(), a, c.ws, c.ws_bytes)
        assert abi.oscar_check_device_error(c.ctx) == 0
        assert c.worst() <= 1.0, bound
    c.close()


def test_one_workspace_for_all_calls_of_a_context_in_turn():
    """Chunks whose keys are split, then single tokens over either cache: the counters stay clear of the records."""
    chunk = Case(8, 2, [(3000, 70, 3070)], -1, 0, False, seed=304)
    others = [Case(8, 2, steps(2500, 20), -1, 0, int4, seed=305) for int4 in (False, True)]
    for _ in range(3):
        for c in (chunk, *others):
            c.ws, c.ws_bytes = chunk.ws, chunk.ws_bytes
            c.out.fill_(9.0)
            c.call()
            assert c.worst() <= 1.0
    for c in (chunk, *others):
        assert abi.oscar_check_device_error(c.ctx) == 0
        c.close()


@pytest.mark.parametrize("int4", [False, True])
def test_two_calls_at_once(int4):
    """One cache and context, two streams, each with a workspace and a result of its own."""
    c = Case(8, 2, steps(4000, 900), -1, 0, int4, seed=306)
    c.check()
    want = c.out.clone()
    streams, outs = [torch.cuda.Stream() for _ in range(2)], [torch.zeros_like(c.out) for _ in range(2)]
    spaces = [torch.zeros_like(c.workspace[0]) for _ in range(2)]
    fn = abi.oscar_window_attention_int4 if int4 else abi.oscar_window_attention_bf16
    torch.cuda.synchronize()
    for _ in range(10):
        for s, out, space in zip(streams, outs, spaces):
            a = c.args()
            a.out = out.data_ptr()
            ws = space.data_ptr() + (-space.data_ptr()) % 256
            fn(c.ctx, c.view(), a, ws, c.ws_bytes, s)
    torch.cuda.synchronize()
    assert abi.oscar_check_device_error(c.ctx) == 0
    for out in outs:
        assert torch.equal(out, want)
    c.close()


def test_the_chunk_next_to_its_first_tokens_alone():
    """A chunk's rows do not depend on how many follow them (beyond the roundings of another split)."""
    c = Case(8, 2, [(500, 64, 564)], -1, 0, False, seed=307)
    c.check()
    whole = f64(c.out)
    c.len.fill_(564)
    a = c.args()
    a.n_tokens, a.max_tokens_per_req = 64, 64
    c.cu[1] = 3
    c.out.fill_(9.0)
    abi.oscar_window_attention_bf16(c.ctx, c.view(), a, c.ws, c.ws_bytes)
    assert abi.oscar_check_device_error(c.ctx) == 0
    assert (c.out[3:] == 9.0).all(), "rows behind the last sequence stay as they were"
    # both are within half a bf16 step of the result, up to the weights' rounding: two tolerances of the oracle's check
    assert np.abs(f64(c.out[:3]) - whole[:3]).max() <= 2 * 2 ** -8 * 2 * np.abs(np.nan_to_num(c.V[0])).max()
    c.close()


def test_a_length_far_beyond_the_host_bound():
    """One request of 1024 claims more than 2^30 / (1024 x 8) tiles: an error and zeros for it, the others as ever."""
    n, Hkv = 1024, 8
    ctx = context(Hkv, Hkv)
    k = torch.randn(1, Hkv, 64, 128, device=DEV).to(torch.bfloat16)
    v = torch.ones_like(k)
    table = torch.zeros(n, (1 << 21) // 64 + 8, dtype=torch.int32, device=DEV)
    q = torch.randn(n, Hkv, 128, device=DEV).to(torch.bfloat16)
    out = torch.full_like(q, 9.0)
    lens = torch.full((n,), 40, dtype=torch.int32, device=DEV)
    pos = lens - 1
    lens[5] = (1 << 21) + 17
    pos[5] = 1 << 21
    _, ws, size = kv.window_workspace(ctx)
    abi.oscar_window_attention_bf16(ctx, kv.bf16_view(k, v, table), kv.window_args(q, out, pos, lens, 64), ws, size)
    assert abi.oscar_check_device_error(ctx) == abi.OSCAR_DEVERR_LENGTH
    assert (out[5] == 0.0).all()
    out[5] = 1.0
    # weights of one sum: fp32 roundings of 40 terms, below half a bf16 step of 1
    assert (out == 1.0).all()
    abi.oscar_destroy(ctx)
