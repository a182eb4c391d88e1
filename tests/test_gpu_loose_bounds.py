"""Host bounds far above the work (a captured step's, a padded batch's) are no error: the same results, bit for bit."""

import numpy as np
import pytest
import torch

from int2_rotated_kv_oscar_gb300 import abi
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
