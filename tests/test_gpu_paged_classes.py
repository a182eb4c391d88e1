"""The cache classes as a program holds them: 4-bit and BF16 pages, filled, attended and read back through their views."""

import numpy as np
import pytest
import torch

from oracle import paged
from int2_rotated_kv_oscar_gb300 import abi
from int2_rotated_kv_oscar_gb300 import cache as kv
from paged_harness import DEV, attention_error, context, f64, int4_rows, ints, rows_of

pytestmark = pytest.mark.gpu


def test_a_4_bit_cache_beside_a_bf16_cache():
    Hq, Hkv, lengths = 8, 2, [150, 0, 65]
    ctx = context(Hq, Hkv)
    codes, plain = kv.Int4PagedCache(Hkv, 8, 3, 3), kv.BF16PagedCache(Hkv, 8, 3, 3)
    table = np.array([[5, 0, 3], [-1, -1, -1], [7, 2, -1]], np.int32)
    codes.page_table.copy_(ints(table))
    plain.page_table.copy_(ints(table))
    n = sum(lengths)
    x = torch.randn(n, Hq + 2 * Hkv, 128, generator=torch.Generator(DEV).manual_seed(1), device=DEV).to(torch.bfloat16)
    q, k, v = x[:, :Hq], x[:, Hq:Hq + Hkv], x[:, Hq + Hkv:]
    cu, zero, lens = ints(np.concatenate([[0], np.cumsum(lengths)])), ints([0, 0, 0]), ints(lengths)
    rope = kv.rope_table(ctx, 256)
    turned, out = torch.empty(n, Hq, 128, dtype=torch.bfloat16, device=DEV), torch.empty(n, Hq, 128, dtype=torch.bfloat16, device=DEV)
    _, ws, size = kv.window_workspace(ctx)
    args = kv.rope_append_args(k, v, zero, q=q, q_out=turned, rope=rope, cu_seqlens=cu, max_tokens_per_req=150)
    look = kv.window_args(turned, out, zero, lens, 150, window=70, sinks=5, cu_seqlens=cu, max_tokens_per_req=150)
    spans = [(0, c, c) for c in lengths]
    abi.oscar_rope_append_int4(ctx, codes.view(), args)
    abi.oscar_window_attention_int4(ctx, codes.view(), look, ws, size)
    assert abi.oscar_check_device_error(ctx) == 0
    K, V, held = [], [], []
    for b, c in enumerate(lengths):
        kc, ks, vc, vs = int4_rows(codes.pages, table, b, c) if c else [np.zeros((0, Hkv, s)) for s in (128, 2, 128, 2)]
        K.append(paged.levels(kc, ks) if c else kc)
        V.append(paged.levels(vc, vs) if c else vc)
        held.append(tuple(s.astype(np.float64).max(-1) if c else np.zeros((0, Hkv)) for s in (ks, vs)))
    assert attention_error(f64(out), f64(turned), K, V, spans, 70, 5, True, held=held) <= 1.0
    # the same tokens in BF16 pages, then the 4-bit cache's rows in their place
    for fill in (lambda: abi.oscar_rope_append_bf16(ctx, plain.view(), args),
                 lambda: abi.oscar_int4_to_bf16(ctx, codes.view(), plain.view(), zero, lens, 150)):
        fill()
        abi.oscar_window_attention_bf16(ctx, plain.view(), look, ws, size)
        assert abi.oscar_check_device_error(ctx) == 0
        rows = [[rows_of(p, table, b, c) for b, c in enumerate(lengths)] for p in (plain.k_pages, plain.v_pages)]
        assert attention_error(f64(out), f64(turned), *rows, spans, 70, 5, False) <= 1.0
    abi.oscar_destroy(ctx)
