"""Attention over packed rows: queries far before position 0, beside a page that is not there."""

import pytest

from test_gpu_prompt import Prompts

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("spans, window, sinks", [
    ([(150, 50), (1, 4000)], -1, 0),       # split keys; a last block of one page
    ([(300, 60), (1, 4000)], 100, 3),
    ([(100, 50), (129, 10), (2, 3000)], -1, 0),
    ([(150, 50), (129, 10)], -1, 0),       # whole items
])
@pytest.mark.parametrize("Hq", [1, 2, 3, 4])
def test_positions_far_before_zero(Hq, spans, window, sinks):
    """Rows up to 240 positions before 0 in one item with rows that see keys: zeros, whatever the page that is not there
    would hold.  (The call before leaves logits of keys that nobody sees, NaN, where that page's would be.)"""
    before = Prompts(Hq, 1, [(60, 300)] * 160, window=30, seed=90)
    before.call()
    c = Prompts(Hq, 1, spans, window, sinks, seed=91)
    for _ in range(3):
        c.check()
        before.call()
    c.close()
    before.close()
