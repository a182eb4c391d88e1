"""Windowed attention at positions next to the largest int32."""

import pytest

from test_gpu_window import Case

pytestmark = pytest.mark.gpu

TOP = 2 ** 31 - 1


@pytest.mark.parametrize("int4", [False, True])
@pytest.mark.parametrize("window, sinks", [(0, 5), (1, 5), (3, 17), (15, 40), (40, 70), (TOP - 300, 5), (TOP - 63, 0), (TOP, 3),
                                           (-1, 0)])
def test_single_tokens_far_out(window, sinks, int4):
    """Far beyond the held positions the first tokens, or what a wide window reaches back to, are all that is seen."""
    spans = [(TOP - 4, 1, 100), (TOP - 1, 1, 40), (TOP, 1, 700), (TOP - 16, 1, 64)]
    c = Case(8, 2, spans, window, sinks, int4, seed=500)
    c.check()
    c.close()


@pytest.mark.parametrize("Hq, Hkv", [(8, 1), (8, 2), (2, 2)])
@pytest.mark.parametrize("window, sinks", [(0, 5), (1, 5), (40, 70), (TOP - 600, 0), (TOP - 600, 66), (TOP - 1000, 3), (TOP, 0),
                                           (-1, 0)])
def test_chunks_far_out(window, sinks, Hq, Hkv):
    for count in (3, 40, 150):
        c = Case(Hq, Hkv, [(TOP - count, count, 1000), (5, 3, 8)], window, sinks, False, seed=501)
        c.check()
        c.close()
