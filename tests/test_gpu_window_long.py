"""4-bit attention whose warps each add up very many keys: what the matrix instructions' sums lose on the way."""

import numpy as np
import pytest
import torch

from oracle import paged, rotation
from int2_rotated_kv_oscar_gb300 import abi
from int2_rotated_kv_oscar_gb300 import cache as kv
from paged_harness import DEV, context, ints

pytestmark = pytest.mark.gpu


def levels(pages, table):
    """fp64 rotated rows [n, 128] of K and V of one KV head's pages [num_pages, 1, 8704] in the table's order."""
    tiles = pages[table.long(), 0].view(-1, paged.TILE_BYTES)
    u, j = np.meshgrid(np.arange(16), np.arange(128), indexing="ij")
    out = []
    for place, scales in ((paged.k_place, 2048), (paged.v_place, 2112)):
        byte, nibble = (torch.from_numpy(np.broadcast_to(x, u.shape).copy()).to(DEV) for x in place(u, j))
        code = (tiles[:, byte.reshape(-1)].view(-1, 16, 128) >> (4 * nibble)) & 15
        s = tiles[:, scales:scales + 64].contiguous().view(torch.float16).view(-1, 16, 2).double()
        out.append(((code.double() - 7.5).view(-1, 16, 2, 64) * s[..., None]).view(-1, 128))
    return out


@pytest.mark.parametrize("Hq", [4, 8])
@pytest.mark.parametrize("requests", [400, 1030])
def test_long_sums(requests, Hq):
    """More (query, KV head) pairs than blocks, of 262,144 keys each (the requests share their pages).

    The limit, of the norm of a row's error: half a bf16 step of the result; six standard deviations of the operands'
    roundings, which are independent (row_errors.py; logits in fp32 add 2^-20 of a weight); and the sums of P V.  A matrix
    instruction truncates what its lane has summed: on average half a step, 2^-24 of a sum that grows evenly, so half of
    that again.  The sums that hold the levels' offset are at most 16 units of two tiles long, 33 instructions, of codes
    up to 15 (bytes up to 255, of which the result takes a sixteenth): 33 2^-25 16 scales, twice that allowed.  The sum
    without the offset goes through n / 128 instructions at about the result's size, twice that allowed."""
    n = 262144
    ctx = context(Hq, 1)
    num = n // 64
    pages = torch.zeros(num, 1, abi.INT4_BLOCK_BYTES, dtype=torch.uint8, device=DEV)
    table = torch.randperm(num, generator=torch.Generator(DEV).manual_seed(3), device=DEV).to(torch.int32)
    x = torch.randn(n, 2, 128, generator=torch.Generator(DEV).manual_seed(1), device=DEV)
    x[:, :, 3] *= 20.0
    x = x.to(torch.bfloat16)
    abi.oscar_rope_append_int4(ctx, kv.int4_view(pages, table[None].contiguous()),
                               kv.rope_append_args(x[:, :1], x[:, 1:], ints([0]), cu_seqlens=ints([0, n])))
    q = (torch.randn(requests, Hq, 128, generator=torch.Generator(DEV).manual_seed(2), device=DEV) * 0.25).to(torch.bfloat16)
    out = torch.full_like(q, 9.0)
    _, ws, size = kv.window_workspace(ctx)
    view = kv.int4_view(pages, table[None].expand(requests, -1).contiguous())
    abi.oscar_window_attention_int4(ctx, view, kv.window_args(q, out, ints([n - 1] * requests), ints([n] * requests), n), ws,
                                    size)
    assert abi.oscar_check_device_error(ctx) == 0
    K, V = levels(pages, table)
    turn = torch.from_numpy(rotation.hadamard(128)).to(DEV).double()
    low = torch.tensor([c for c in range(128) if not c & 2], device=DEV)
    scale = 128 ** -0.5
    top = float(V.abs().max() / 7.5)
    for r in (0, requests // 3, requests - 1):
        for h in (0, Hq - 1):
            qr = q[r, h].double() @ turn
            w = torch.softmax(K @ qr * scale, 0)
            o = w @ V
            d = V - o
            half = 2.0 ** -16 if Hq <= 4 else 2.0 ** -8
            var = (w ** 2 * (half ** 2 / 3 * (V ** 2).sum(1) + 2.0 ** -38 * (d ** 2).sum(1))).sum()
            if Hq > 4:
                m = (K * w[:, None] * scale).T @ d
                h1 = qr[low + 2] / 16
                h0 = qr[low] - h1
                var += 2.0 ** -22 / 3 * ((h0 ** 2 * (m[low] ** 2).sum(1)).sum()
                                         + (h1 ** 2 * ((m[low] + 16 * m[low + 2]) ** 2).sum(1)).sum())
            sums = 2 * 33 * 2.0 ** -25 * 16 * top * 128 ** 0.5 + 2 * n / 128 * 2.0 ** -24 * float(o.norm())
            limit = 2.0 ** -8 * float(o.norm()) + 6 * float(var) ** 0.5 + sums
            error = float((out[r, h].double() @ turn - o).norm())
            assert error <= limit, (r, h, error / float(o.norm()), limit / float(o.norm()))
    abi.oscar_destroy(ctx)
