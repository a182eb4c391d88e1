"""A query that is not finite gives NaN, whichever kernel attends, and leaves the others alone."""

import numpy as np
import pytest

from test_gpu_window import Case, steps
from paged_harness import f64

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("value", [float("nan"), float("inf"), float("-inf")])
@pytest.mark.parametrize("spans, int4", [(steps(3000, 70, 900), False), (steps(3000, 70, 900), True), ([(4000, 40, 4040)], False),
                                         ([(0, 300, 300), (20, 40, 60)], False), ([(500, 5, 505)], True)])
def test_queries_that_are_not_finite(spans, int4, value):
    c = Case(8, 2, spans, -1, 0, int4, seed=600)
    row, head = c.n // 2, 5
    clean = c.q[row, head].clone()
    c.call()
    want = f64(c.out)
    c.q[row, head, 3] = value  # its logits: NaN, or infinities of both signs
    c.out.fill_(9.0)
    c.call()
    got = f64(c.out)
    assert np.isnan(got[row, head]).all()
    got[row, head] = want[row, head]
    # a KV head's other queries share its products' tiles but no sum with this one
    assert np.array_equal(got, want)
    c.q[row, head] = clean
    c.check()
    c.close()
