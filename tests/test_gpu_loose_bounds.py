"""Host bounds far above the work (a captured step's, a padded batch's) are no error: the same results, bit for bit."""

import numpy as np
import pytest
import torch

from int2_rotated_kv_oscar_gb300 import abi
from int2_rotated_kv_oscar_gb300 import cache as kv
from paged_harness import DEV, context, ints
from test_gpu_read2 import Held

pytestmark = pytest.mark.gpu


def test_read_back():
    lengths = [int(n) for n in np.random.default_rng(9).integers(0, 700, 64)]
    h = Held(8, lengths, seed=30)
    h.read([0] * 64, lengths)
    want = h.k_pages.clone(), h.v_pages.clone()
    for most in (2 ** 28, 2 ** 31 - 1):
        h.k_pages.fill_(float("nan"))
        h.v_pages.fill_(float("nan"))
        h.read([0] * 64, lengths, most=most)
        assert abi.oscar_check_device_error(h.ctx) == 0
        for got, ref in zip((h.k_pages, h.v_pages), want):
            assert torch.equal(got.view(torch.int16), ref.view(torch.int16))
    h.close()


def test_prompt_attention():
    """65,535 requests, three of which have tokens, among 140,000 rows, with the rows as the bound of a request's tokens."""
    Hq, Hkv, n, B = 64, 8, 140_000, 65535
    r = torch.Generator(device=DEV).manual_seed(31)
    q, k, v = [torch.randn(n, h, 128, generator=r, device=DEV, dtype=torch.bfloat16) for h in (Hq, Hkv, Hkv)]
    cu = np.full(B + 1, 340, np.int32)
    cu[:20000], cu[20000:65535] = 0, 300
    cu[50000:65535] = 333
    ctx = context(Hq, Hkv)
    _, ws, size = workspace = kv.window_workspace(ctx)
    want, got = torch.full_like(q, 9), torch.full_like(q, 9)
    abi.oscar_prompt_attention(ctx, kv.prompt_args(q, k, v, want, ints(cu), 300), ws, size)
    abi.oscar_prompt_attention(ctx, kv.prompt_args(q, k, v, got, ints(cu), n), ws, size)
    assert abi.oscar_check_device_error(ctx) == 0
    assert torch.equal(got, want) and (got[340:] == 9).all() and not (got[:340] == 9).all()
    del workspace
    abi.oscar_destroy(ctx)
