"""Integers that the ABI's 32 bits do not hold are refused, never wrapped into another number (2^32 is no 0)."""

import numpy as np
import pytest
import torch

from int2_rotated_kv_oscar_gb300 import abi, build
from int2_rotated_kv_oscar_gb300 import cache as kv

BAD = [2 ** 31, 2 ** 32, 2 ** 32 + 5, -2 ** 31 - 1]


@pytest.fixture(scope="module", autouse=True)
def lib():
    build.build()
    return abi.load(build_if_missing=False)


def ints(n):
    return torch.zeros(n, dtype=torch.int32)


def calls():
    """name -> (function of one integer); no context, so that what gets past the check is the library's refusal."""
    mixed = kv.MixedCache(1, 2, 3, 2, 2, 2, 3, device="cpu")
    pool = torch.zeros(3, 2, 64, 128, dtype=torch.bfloat16)
    to = kv.bf16_view(pool, pool.clone(), torch.zeros(2, 3, dtype=torch.int32))
    four = kv.Int4PagedCache(2, 3, 2, 3, device="cpu").view()
    view, i, u = mixed.view(0), ints(2), np.eye(128, dtype=np.float32)
    new, q = abi.oscar_append_args(), abi.oscar_decode_args()
    out = {
        "load": lambda x: abi.oscar_load_rotation(None, x, u, u, 1.0, 1.0),
        "append": lambda x: abi.oscar_kv_append(None, x, view, new),
        "decode": lambda x: abi.oscar_decode_attention(None, x, view, q, None, 0),
        "extend": lambda x: abi.oscar_extend_attention(None, x, view, q, None, None, 0),
        "step": lambda x: abi.oscar_decode_step(None, x, view, new, q, None, 0),
        "noalloc": lambda x: abi.oscar_decode_attention_noalloc(None, x, view, q),
        "read layer": lambda x: abi.oscar_int2_to_bf16(None, x, view, to, i, i, i, 4),
        "read count": lambda x: abi.oscar_int2_to_bf16(None, 0, view, to, i, i, i, x),
        "read 4 bits": lambda x: abi.oscar_int4_to_bf16(None, four, to, i, i, x),
        "threshold": lambda x: abi.oscar_calib_clip_threshold(None, None, x, u, 7, 99.9, None, 0),
    }
    for at in range(3):
        def chunk(x, at=at):
            layer, n, most = [x if k == at else 1 for k in range(3)]
            abi.oscar_extend_chunk(None, layer, view, None, None, None, None, n, most, None, 0)

        def covariances(x, at=at):
            n_q, n_k, heads = [x if k == at else 1 for k in range(3)]
            abi.oscar_calib_covariances(None, None, n_q, None, None, n_k, heads, 1.0, None, None, None, 0)

        out["chunk %d" % at], out["covariances %d" % at] = chunk, covariances
    return out


NAMES = sorted(calls())


@pytest.mark.parametrize("name", NAMES)
def test_calls(name):
    call = calls()[name]
    for x in BAD:
        with pytest.raises(ValueError):
            call(x)
    with pytest.raises(abi.OscarError):  # one that fits reaches the library, which refuses the missing context
        call(1)


def test_sizes():
    for fn, n in ((lambda *a: abi.oscar_decode_workspace_bytes(None, *a), 2),
                  (lambda *a: abi.oscar_extend_workspace_bytes(None, *a), 3), (abi.oscar_calib_workspace_bytes, 4)):
        for at in range(n):
            for x in BAD:
                with pytest.raises(ValueError):
                    fn(*[x if k == at else 1 for k in range(n)])


def test_helpers():
    q, k = torch.zeros(2, 4, 128, dtype=torch.bfloat16), torch.zeros(2, 2, 128, dtype=torch.bfloat16)
    for x in BAD:
        for make in (lambda: kv.append_args(k, k, ints(2), max_tokens_per_req=x),
                     lambda: kv.decode_args(q, q.float(), ints(2), x),
                     lambda: kv.rope_append_args(k, k.clone(), ints(2), max_tokens_per_req=x),
                     lambda: kv.window_args(q, q.clone(), ints(2), ints(2), x),
                     lambda: kv.window_args(q, q.clone(), ints(2), ints(2), 5, window=x),
                     lambda: kv.window_args(q, q.clone(), ints(2), ints(2), 5, sinks=x),
                     lambda: kv.window_args(q, q.clone(), ints(2), ints(2), 5, cu_seqlens=ints(3), max_tokens_per_req=x)):
            with pytest.raises(ValueError):
                make()
