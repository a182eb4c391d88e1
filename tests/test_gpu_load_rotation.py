"""oscar_load_rotation: a layer is complete when it returns, so that a read-back at once, on a stream that does not wait for
the default one, sees all of it (also a layer that is loaded again); entries of any size."""

import numpy as np
import pytest
import torch

from int2_rotated_kv_oscar_gb300 import abi
from oracle import rotation
from test_gpu_read2 import Held

pytestmark = pytest.mark.gpu


def test_read_back_right_behind_a_load():
    h = Held(2, [500, 700], seed=3)
    r = np.random.default_rng(4)
    us = [np.linalg.qr(r.standard_normal((128, 128)))[0].astype(np.float32) for _ in range(2)]

    def read(u, wait):
        abi.oscar_load_rotation(h.ctx, 0, u, u, 20.0, 30.0)
        if wait:
            torch.cuda.synchronize()
        h.read([0, 0], [500, 700])

    side = torch.cuda.Stream()
    want = []
    with torch.cuda.stream(side):
        for u in us:
            read(u, True)
            side.synchronize()
            want.append((h.k_pages.clone(), h.v_pages.clone()))
        for i in range(40):
            h.k_pages.fill_(float("nan"))
            h.v_pages.fill_(float("nan"))
            side.synchronize()
            read(us[i % 2], False)
            side.synchronize()
            for got, ref in zip((h.k_pages, h.v_pages), want[i % 2]):
                see = ~torch.isnan(ref)
                assert torch.equal(got[see], ref[see])
    assert abi.oscar_check_device_error(h.ctx) == 0
    h.close()


@pytest.mark.parametrize("flags", [abi.OSCAR_ROT_U, abi.OSCAR_ROT_ALL])
@pytest.mark.parametrize("scale", [3000.0, 1.0, 2.0 ** -13, 1e-6])
def test_entries_of_any_size(scale, flags):
    """R's two fp16 terms above, around and below the smallest normal number (2^-14), by the read-back's bounds."""
    h = Held(2, [500, 700], seed=5, flags=flags)
    u = [(np.random.default_rng(k).standard_normal((128, 128)) * scale).astype(np.float32) for k in (6, 7)]
    abi.oscar_load_rotation(h.ctx, 0, u[0], u[1], 20.0, 30.0, flags)
    h.R = [[rotation.composite_rotation(x.astype(np.float64), *[bool(flags & f) for f in (1, 2, 4)]) for x in u]]
    h.read([0, 0], [500, 700])
    h.check([0, 0], [500, 700])
    h.close()
