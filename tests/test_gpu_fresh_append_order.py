"""The mixed cache's append of a fresh prompt behind kernels of this library that let the next one start early."""

import numpy as np
import pytest
import torch

from int2_rotated_kv_oscar_gb300 import abi
from int2_rotated_kv_oscar_gb300 import cache as kv
from paged_harness import DEV, context, ints, nan_int4, nan_pages

pytestmark = pytest.mark.gpu


def mixed_cache(ctx, Hkv, n):
    eye = np.eye(128, dtype=np.float32)
    abi.oscar_load_rotation(ctx, 0, eye, eye, 1.0, 1.0)
    pages = n // 64 + 2
    mixed = kv.MixedCache(1, Hkv, pages, 1, 1, 1, pages)
    mixed.page_table.copy_(torch.arange(pages, device=DEV, dtype=torch.int32)[None])
    return mixed


def bf16_rows_match(mixed, k, v, n):
    """The sink's and the ring's rows are those of k and v [n, Hkv, 128]."""
    at = torch.arange(max(n - 256, 64), n, device=DEV)
    for rows, ring, sink in ((k, mixed.k_ring[0][0], mixed.k_sink[0][0]), (v, mixed.v_ring[0][0], mixed.v_sink[0][0])):
        assert torch.equal(ring[:, (at - 64) % 256].transpose(0, 1), rows[at])
        assert torch.equal(sink.transpose(0, 1), rows[:64])


@pytest.mark.parametrize("n", [320, 700, 6000, 40000])
def test_rows_read_back_feed_the_mixed_cache_at_once(n):
    """With one KV head the pages that a read-back fills, in order, are the packed K and V of an append."""
    ctx = context(1, 1)
    mixed = mixed_cache(ctx, 1, n)
    num = -(-n // 64)
    table = torch.arange(num, device=DEV, dtype=torch.int32)[None]
    pages = nan_int4(num, 1)
    pos, cu, count = ints([0]), ints([0, n]), ints([n])
    for i in range(8):
        x = torch.randn(n, 2, 128, generator=torch.Generator(DEV).manual_seed(i), device=DEV).to(torch.bfloat16)
        k_pages, v_pages = nan_pages(num, 1)
        k, v = (p.view(-1, 1, 128)[:n] for p in (k_pages, v_pages))
        args = kv.append_args(k, v, pos, cu_seqlens=cu, fresh_ring=True)
        abi.oscar_rope_append_int4(ctx, kv.int4_view(pages, table), kv.rope_append_args(x[:, :1], x[:, 1:], pos, cu_seqlens=cu))
        view4, view = kv.int4_view(pages, table), kv.bf16_view(k_pages, v_pages, table)
        torch.cuda.synchronize()
        abi.oscar_int4_to_bf16(ctx, view4, view, pos, count, n)
        abi.oscar_kv_append(ctx, 0, mixed.view(0), args)
        assert abi.oscar_check_device_error(ctx) == 0
        assert torch.isfinite(k.float()).all() and torch.isfinite(v.float()).all()
        bf16_rows_match(mixed, k, v, n)
    abi.oscar_destroy(ctx)


@pytest.mark.parametrize("tokens", [1, 400])
def test_an_attention_result_feeds_the_mixed_cache_at_once(tokens):
    """With as many KV heads as query heads the result [n, H, 128] of an attention can be an append's K and V."""
    H, held = 2, 3000
    n = 400
    ctx = context(H, H)
    mixed = mixed_cache(ctx, H, n)
    num = -(-held // 64)
    pools = [torch.randn(num, H, 64, 128, generator=torch.Generator(DEV).manual_seed(s), device=DEV).to(torch.bfloat16)
             for s in (1, 2)]
    q = torch.randn(n, H, 128, generator=torch.Generator(DEV).manual_seed(3), device=DEV).to(torch.bfloat16)
    requests = n // tokens
    table = torch.arange(num, device=DEV, dtype=torch.int32)[None].expand(requests, -1).contiguous()
    pos = ints([held - tokens - (i if tokens == 1 else 0) for i in range(requests)])
    lens = ints([held] * requests)
    cu = None if tokens == 1 else ints([0, n])
    _, ws, size = kv.window_workspace(ctx)
    view = kv.bf16_view(*pools, table)
    for _ in range(6):
        out = torch.full_like(q, float("nan"))
        attend = kv.window_args(q, out, pos, lens, held, cu_seqlens=cu)
        args = kv.append_args(out, out, ints([0]), cu_seqlens=ints([0, n]), fresh_ring=True)
        torch.cuda.synchronize()
        abi.oscar_window_attention_bf16(ctx, view, attend, ws, size)
        abi.oscar_kv_append(ctx, 0, mixed.view(0), args)
        assert abi.oscar_check_device_error(ctx) == 0
        assert torch.isfinite(out.float()).all()
        bf16_rows_match(mixed, out, out, n)
    abi.oscar_destroy(ctx)
