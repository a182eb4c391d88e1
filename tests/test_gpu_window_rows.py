"""Windowed attention, row by row: a limit on each row's error that no missing key, mask or constant gets past."""

import pytest

from int2_rotated_kv_oscar_gb300 import abi
from row_errors import row_errors
from test_gpu_window import Case, steps
from paged_harness import f64

pytestmark = pytest.mark.gpu

TOKENS = [
    dict(Hq=16, Hkv=2, spans=steps(700, 33, 64, 129), window=65, sinks=70),
    dict(Hq=8, Hkv=1, spans=steps(5003), window=-1, sinks=0),
    dict(Hq=8, Hkv=1, spans=steps(700, 1, 300), window=-1, sinks=0),
    dict(Hq=5, Hkv=1, spans=steps(300, 2, 77), window=0, sinks=5),
    dict(Hq=6, Hkv=1, spans=steps(257, 1024), window=100, sinks=40),
    dict(Hq=8, Hkv=2, spans=steps(1, 5, 70, 500, 1000), window=7, sinks=3),
    dict(Hq=4, Hkv=4, spans=steps(1500, 90, 260), window=200, sinks=64),
    dict(Hq=32, Hkv=4, spans=steps(*range(90, 1200, 61)), window=-1, sinks=0),
    dict(Hq=4, Hkv=1, spans=[(100, 1, 95), (40, 1, 200), (2000, 1, 2001)], window=33, sinks=17),
]

CHUNKS = [
    dict(Hq=8, Hkv=1, spans=[(300, 70, 370), (0, 1, 1)], window=100, sinks=64),
    dict(Hq=8, Hkv=2, spans=[(0, 5, 5), (60, 9, 69), (700, 20, 720)], window=-1, sinks=0),
    dict(Hq=5, Hkv=1, spans=[(10, 60, 70)], window=16, sinks=0),
    dict(Hq=8, Hkv=1, spans=[(3000, 17, 3017)], window=-1, sinks=0),
    dict(Hq=6, Hkv=1, spans=[(130, 65, 195)], window=64, sinks=130),
]


def check(c):
    c.call()
    assert abi.oscar_check_device_error(c.ctx) == 0
    pack = c.Hq // c.Hkv <= 4 and (c.single or c.int4)
    assert row_errors(f64(c.out), f64(c.q), c.K, c.V, c.spans, c.window, c.sinks, pack, held=c.held,
                      tensor_cores=not c.int4 and not c.single) <= 1.0
    c.close()


@pytest.mark.parametrize("int4", [False, True])
@pytest.mark.parametrize("q_scale", [0.25, 1.0])
@pytest.mark.parametrize("i", range(len(TOKENS)))
def test_rows_of_single_tokens(i, q_scale, int4):
    check(Case(**TOKENS[i], int4=int4, seed=700 + i, q_scale=q_scale))


@pytest.mark.parametrize("int4", [False, True])
@pytest.mark.parametrize("q_scale", [0.25, 1.0])
@pytest.mark.parametrize("i", range(len(CHUNKS)))
def test_rows_of_chunks(i, q_scale, int4):
    check(Case(**CHUNKS[i], int4=int4, seed=720 + i, q_scale=q_scale))
