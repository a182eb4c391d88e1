"""A query whose logits are all -infinity is not finite, and gives NaN as such; one that sees nothing gives zeros."""

import numpy as np
import pytest
import torch

from int2_rotated_kv_oscar_gb300 import abi
from oracle import paged
from paged_harness import attention_error, f64
from row_errors import row_errors
from test_gpu_prompt import Prompts, whole
from test_gpu_window import Case, steps

pytestmark = pytest.mark.gpu


def check(c, out, q, rows, head, tensor_cores):
    """Head `head` of the rows named is poisoned: NaN, or zeros where the row sees nothing.  The others keep to their bounds."""
    got, i = f64(out), 0
    for b, (p0, count, ctx) in enumerate(c.spans):
        for p in range(p0, p0 + count):
            if i in rows:
                sees = paged.visible(p, ctx, c.window, c.sinks).any()
                assert np.isnan(got[i, head]).all() if sees else not got[i, head].any(), (b, p)
                h = head // (c.Hq // c.Hkv)
                got[i, head] = paged.attend(q[i, head], c.K[b][:ctx, h], c.V[b][:ctx, h], p, c.window, c.sinks, 128 ** -0.5)[0]
            i += 1
    pack = c.Hq // c.Hkv <= 4 and not tensor_cores
    assert attention_error(got, q, c.K, c.V, c.spans, c.window, c.sinks, pack) <= 1.0
    assert row_errors(got, q, c.K, c.V, c.spans, c.window, c.sinks, pack, tensor_cores=tensor_cores) <= 1.0


@pytest.mark.parametrize("value", [float("inf"), float("-inf")])
@pytest.mark.parametrize("Hq, Hkv", [(8, 2), (3, 1), (8, 1)])
@pytest.mark.parametrize("spans, window, sinks, rows", [
    (whole(1), -1, 0, [0]), (whole(300, 60), -1, 0, [0, 1, 130, 299, 300]), (whole(300), 40, 3, [0, 150, 299]),
    (whole(90), 0, 2, [0, 50]), ([(40, 4040)], -1, 0, [0, 39]), ([(1, 3000), (20, 10)], -1, 0, [0, 1, 11, 20]),
    ([(40, 900)], 200, 0, [0, 39]), ([(100, 30), (9, 0)], -1, 0, [0, 69, 70, 99, 104])])
def test_packed_rows(Hq, Hkv, spans, window, sinks, rows, value):
    c = Prompts(Hq, Hkv, spans, window, sinks, seed=95)
    c.k[:, :, 3] = -torch.sign(torch.tensor(value)) * (c.k[:, :, 3].abs() + 1)  # every key against the query's channel
    at = c.lead
    for b, (_, _, nk) in enumerate(c.spans):
        c.K[b] = f64(c.k[at:at + nk])
        at += nk
    head = Hq - 1
    clean = c.q.clone()
    for r in rows:
        c.q[c.lead + r, head, 3] = value
    c.call()
    assert abi.oscar_check_device_error(c.ctx) == 0
    check(c, c.out[c.lead:-2], f64(clean[c.lead:-2]), rows, head, True)
    c.close()


CHUNKS = [([(0, 5, 5), (60, 9, 69)], -1, 0, [0, 4, 5]), ([(0, 200, 200)], 50, 4, [0, 150]),
          ([(0, 90, 60), (100, 40, 95)], 20, 0, [0, 89, 90, 129]), ([(4000, 40, 4040)], -1, 0, [0, 39])]


def over_pages(Hq, Hkv, spans, window, sinks, rows, value):
    c = Case(Hq, Hkv, spans, window, sinks, False, seed=96)
    sign = -float(np.sign(value))
    c.k_pages[..., 3] = sign * (c.k_pages[..., 3].abs() + 1)
    for k in c.K:
        k[:, :, 3] = f64(torch.from_numpy(sign * (np.abs(k[:, :, 3]) + 1)).to(torch.bfloat16))
    head = Hq - 1
    clean = f64(c.q)
    for r in rows:
        c.q[r, head, 3] = value
    c.call()
    assert abi.oscar_check_device_error(c.ctx) == 0
    check(c, c.out, clean, rows, head, not c.single)
    c.close()


@pytest.mark.parametrize("value", [float("inf"), float("-inf")])
@pytest.mark.parametrize("Hq, Hkv", [(8, 2), (3, 1), (8, 1)])
@pytest.mark.parametrize("spans, window, sinks, rows", CHUNKS)
def test_chunks_over_pages(Hq, Hkv, spans, window, sinks, rows, value):
    over_pages(Hq, Hkv, spans, window, sinks, rows, value)


@pytest.mark.parametrize("count, ctx", [(40, 40), (20, 3000)])  # whole items, split ones
def test_chunks_that_see_bad_pages_alone(count, ctx):
    """Positions of pages outside the pool are left out, so that nothing is left to see."""
    c = Case(4, 1, [(ctx - count, count, ctx), (0, 30, 30)], -1, 0, False, seed=97)
    c.pt[0].fill_(1 << 30)
    c.q[:, 3, 3] = float("-inf")
    c.k_pages[..., 3] = c.k_pages[..., 3].abs() + 1
    c.call()
    assert abi.oscar_check_device_error(c.ctx) == abi.OSCAR_DEVERR_PAGE
    assert not c.out[:count].any()
    assert torch.isnan(c.out[count:, 3]).all() and not torch.isnan(c.out[count:, :3]).any()
    c.close()


@pytest.mark.parametrize("value", [float("inf"), float("-inf")])
@pytest.mark.parametrize("Hq, Hkv", [(8, 2), (3, 1), (8, 1)])
@pytest.mark.parametrize("spans, window, sinks, rows", [
    (steps(1, 2, 70, 900), -1, 0, [0, 1, 3]), (steps(3000, 40), 100, 3, [0, 1]), (steps(20011), -1, 0, [0]),
    ([(0, 1, 0), (40, 1, 41), (100, 1, 50)], 10, 0, [0, 1, 2])])
def test_tokens_over_pages(Hq, Hkv, spans, window, sinks, rows, value):
    over_pages(Hq, Hkv, spans, window, sinks, rows, value)


@pytest.mark.parametrize("value", [float("inf"), float("-inf")])
@pytest.mark.parametrize("Hq, Hkv", [(8, 2), (8, 1)])
def test_tokens_over_4_bits(Hq, Hkv, value):
    c = Case(Hq, Hkv, steps(1, 2, 300), -1, 0, True, seed=98)
    c.q[:, 2, 3] = value
    c.call()
    assert abi.oscar_check_device_error(c.ctx) == 0
    assert torch.isnan(c.out[:, 2]).all()
    rest = [h for h in range(Hq) if h != 2]
    assert not torch.isnan(c.out[:, rest]).any()
    c.close()


@pytest.mark.parametrize("ctx", [30, 5000])  # one block's, and cut into several
def test_tokens_that_see_bad_pages_alone(ctx):
    c = Case(4, 1, steps(ctx, 30), -1, 0, False, seed=99)
    c.pt[0].fill_(1 << 30)
    c.q[:, 3, 3] = float("-inf")
    c.k_pages[..., 3] = c.k_pages[..., 3].abs() + 1
    c.call()
    assert abi.oscar_check_device_error(c.ctx) == abi.OSCAR_DEVERR_PAGE
    assert not c.out[0].any()
    assert torch.isnan(c.out[1, 3]).all() and not torch.isnan(c.out[1, :3]).any()
    c.close()
