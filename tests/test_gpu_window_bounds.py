"""Single tokens whose launch is larger than their work: host bounds far above the lengths, batches of nearly empty slots."""

import pytest
import torch

from int2_rotated_kv_oscar_gb300 import abi
from test_gpu_window import Case, steps

pytestmark = pytest.mark.gpu


def attend(c, bound):
    a = c.args()
    a.max_ctx_len = bound
    c.out.fill_(9.0)
    fn = abi.oscar_window_attention_int4 if c.int4 else abi.oscar_window_attention_bf16
    fn(c.ctx, c.view(), a, c.ws, c.ws_bytes)
    assert abi.oscar_check_device_error(c.ctx) == 0
    assert c.worst() <= 1.0, bound


def counters(c):
    """The words at the workspace's start that blocks of one result count in (two for each SM)."""
    tensor, at, _ = c.workspace
    at -= tensor.data_ptr()
    return tensor[at:at + 8 * abi.oscar_device_sm_count(c.ctx)]


@pytest.mark.parametrize("int4", [False, True])
@pytest.mark.parametrize("Hq, Hkv", [(1, 1), (8, 1), (8, 2), (16, 4), (24, 3)])
@pytest.mark.parametrize("length", [18, 288, 290, 480, 515, 577, 1000, 1184, 2000, 2368])
def test_host_bounds_above_the_lengths(length, Hq, Hkv, int4):
    """A graph of a decode step keeps the engine's largest length as its bound; each call leaves the workspace usable."""
    c = Case(Hq, Hkv, steps(length), -1, 0, int4, seed=400)
    for bound in (length, 4 * length, 32 * length, 128 * length, 1 << 20, length):
        attend(c, bound)
        assert not counters(c).any(), bound
    c.close()


@pytest.mark.parametrize("int4", [False, True])
@pytest.mark.parametrize("Hq, Hkv, live, others", [(8, 8, 1024, [0] * 63), (16, 4, 1280, [0] * 31), (4, 1, 3200, [32] * 63),
                                                   (8, 1, 1600, [16] * 39), (8, 2, 700, [0, 5] * 20 + [300])])
def test_one_long_request_among_short_ones(Hq, Hkv, live, others, int4):
    """A padded decode batch: the bound is exact for one request and far above the others."""
    for at in (0, len(others) // 2):
        lengths = others[:at] + [live] + others[at:]
        c = Case(Hq, Hkv, [(max(n - 1, 0), 1, n) for n in lengths], -1, 0, int4, seed=401)
        for bound in (live, 32 * live, live):
            attend(c, bound)
            assert not counters(c).any(), bound
        c.close()


@pytest.mark.parametrize("int4", [False, True])
@pytest.mark.parametrize("Hq, Hkv", [(4, 1), (16, 2)])
def test_a_captured_step_while_the_lengths_grow(Hq, Hkv, int4):
    """Captured once with the largest length as the bound, replayed from the first token on."""
    total = 1500
    c = Case(Hq, Hkv, steps(total), -1, 0, int4, seed=402)
    a = c.args()
    a.max_ctx_len = 131072
    fn = abi.oscar_window_attention_int4 if int4 else abi.oscar_window_attention_bf16
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        fn(c.ctx, c.view(), a, c.ws, c.ws_bytes, torch.cuda.current_stream())
    for n in (1, 14, 40, 79, 257, 300, 513, 800, 1100, total):
        c.pos.fill_(n - 1)
        c.len.fill_(n)
        c.spans = steps(n)
        c.out.fill_(9.0)
        graph.replay()
        torch.cuda.synchronize()
        assert abi.oscar_check_device_error(c.ctx) == 0
        assert c.worst() <= 1.0, n
        assert not counters(c).any(), n
    c.close()
