"""Weights that add up over many keys without a block of keys that stands out: V up to 2^77 does not overflow.

Every key's logit is the same, about 33.9 in base 2 above the reference, so that no half block's sum reaches 2^40; all V
rows are one row, which is then the result: off by a weight's rounding and the result's own (2^-8 each), and 2^-23 for
each 16 keys' step of the tensor cores' sums (truncated, of P V and l alike)."""

import numpy as np
import pytest
import torch

from int2_rotated_kv_oscar_gb300 import abi
from int2_rotated_kv_oscar_gb300 import cache as kv
from paged_harness import DEV, context, f64, ints

pytestmark = pytest.mark.gpu

BITS = 33.9
N = 300_000


def rows(n, heads, value):
    x = torch.zeros(n, heads, 128, dtype=torch.bfloat16, device=DEV)
    x[..., 0] = value
    return x


def setup(tokens, Hq):
    q = rows(tokens, Hq, 16.0)
    k = rows(N, 1, BITS * np.log(2.0) * 128 ** 0.5 / 16)
    r = np.random.default_rng(5)
    row = torch.from_numpy(r.choice([-1.0, 1.0], 128) * 2.0 ** r.uniform(76.0, 77.0, 128)).to(DEV, torch.bfloat16)
    return q, k, row.expand(N, 1, 128).contiguous(), row


def check(out, row):
    want = f64(row)
    tol = (2 * 2.0 ** -8 + N / 16 * 2.0 ** -23) * np.abs(want)
    for at in range(0, out.shape[0], 1024):
        assert (np.abs(f64(out[at:at + 1024]) - want) <= tol).all()


@pytest.mark.parametrize("tokens", [1, 40, 9728])  # split keys, and whole items of all of them
def test_packed_rows(tokens):
    ctx = context(8, 1)
    q, k, v, row = setup(tokens, 8)
    out = torch.empty_like(q)
    _, ws, size = workspace = kv.window_workspace(ctx)
    abi.oscar_prompt_attention(ctx, kv.prompt_args(q, k, v, out, ints([0, tokens]), tokens, cu_seqlens_k=ints([0, N]),
                                                   max_keys_per_req=N), ws, size)
    assert abi.oscar_check_device_error(ctx) == 0
    check(out, row)
    del workspace
    abi.oscar_destroy(ctx)


@pytest.mark.parametrize("tokens", [40, 9728])
def test_pages(tokens):
    """The reference is the first block's maximum, a logit of 0; the other keys weigh as above."""
    ctx = context(8, 1)
    q, k, v, row = setup(tokens, 8)
    k[:128, :, 0] = 0.0
    out = torch.empty_like(q)
    n_pages = (N + 63) // 64
    k_pages, v_pages = [torch.nn.functional.pad(x[:, 0], (0, 0, 0, 64 * n_pages - N)).view(n_pages, 1, 64, 128) for x in (k, v)]
    _, ws, size = workspace = kv.window_workspace(ctx)
    abi.oscar_window_attention_bf16(ctx, kv.bf16_view(k_pages, v_pages, ints([list(range(n_pages))])),
                                    kv.window_args(q, out, ints([N - tokens]), ints([N]), N, cu_seqlens=ints([0, tokens]),
                                                   max_tokens_per_req=tokens), ws, size)
    assert abi.oscar_check_device_error(ctx) == 0
    check(out, row)
    del workspace
    abi.oscar_destroy(ctx)
