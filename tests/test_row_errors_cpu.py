"""The row check itself: the kernels' roundings pass it, single mistakes do not."""

import numpy as np
import pytest
import torch

from oracle import paged
from row_errors import row_errors


def bf16(x):
    return torch.from_numpy(np.asarray(x, np.float32)).to(torch.bfloat16).double().numpy()


class Rows:
    """One query group of one KV head over n keys, in 4 bits or BF16, and the result with the kernel's roundings."""

    def __init__(self, g, n, window, sinks, int4, seed, q_scale):
        r = np.random.default_rng([seed, g, n])
        self.g, self.n, self.window, self.sinks, self.int4 = g, n, window, sinks, int4
        rows = r.standard_normal((2, n, 128))
        rows[:, :, 3] *= 20.0
        rows = bf16(rows)
        self.q = bf16(r.standard_normal((1, g, 128)) * q_scale)
        if int4:
            (kc, ks, _), (vc, vs, _) = (paged.quantise(paged.to_rotated(x)) for x in rows)
            self.codes = kc, ks, vc, vs
            self.k, self.v = paged.levels(kc, ks), paged.levels(vc, vs)
            self.held = [(ks.astype(np.float64).max(-1)[:, None], vs.astype(np.float64).max(-1)[:, None])]
        else:
            self.k, self.v, self.held = rows[0], rows[1], None

    def result(self, see=None, k_offset=7.5, v_offset=7.5, k_scale=(1.0, 1.0), head=None):
        """The kernel's operands: fp16 queries and one bf16 weight a key for g > 4, else two terms of each."""
        pack = self.g <= 4
        see = paged.visible(self.n - 1, self.n, self.window, self.sinks) if see is None else see
        out = np.zeros((1, self.g, 128))
        for h in range(self.g):
            q = self.q[0, h if head is None else head]
            if self.int4:
                kc, ks, vc, vs = (x[see].astype(np.float64) for x in self.codes)
                qr = paged.to_rotated(q)
                low = np.array([c for c in range(128) if not c & 2])
                up = 2.0 ** (14 - np.floor(np.log2(np.abs(qr).max())))
                ops = [(qr[low] - qr[low + 2] / 16) * up, qr[low + 2] / 16 * up]
                h0, h1 = (np.float16(x).astype(np.float64) for x in ops)
                if pack:
                    h0, h1 = ops
                terms = np.zeros((kc.shape[0], 128))
                terms[:, low] = (h0 + h1) * (kc[:, low] - k_offset)
                terms[:, low + 2] = 16 * h1 * (kc[:, low + 2] - k_offset)
                x = sum(terms[:, 64 * i:64 * i + 64].sum(1) * ks[:, i] * k_scale[i] for i in range(2)) / up
            else:
                kc = self.k[see]
                x = kc @ q
            x = x * 128 ** -0.5
            p = np.exp(x - x.max())
            if self.int4:
                w = [p * vs[:, i] for i in range(2)]
                w = [y if pack else bf16(y) for y in w]
                o = np.concatenate([w[i] @ (vc[:, 64 * i:64 * i + 64] - v_offset) for i in range(2)])
                o = paged.from_rotated(o / p.sum())
            else:
                o = (p if pack else bf16(p)) @ self.v[see] / p.sum()
            out[0, h] = bf16(o)
        return out

    def worst(self, out):
        return row_errors(out, self.q, [self.k[:, None]], [self.v[:, None]], [(self.n - 1, 1, self.n)], self.window, self.sinks,
                          self.g <= 4, held=self.held)


CASES = [(8, 700, 65, 70), (8, 700, -1, 0), (5, 300, -1, 0), (8, 5003, -1, 0), (4, 1000, -1, 0), (4, 700, 65, 70), (1, 5003, -1, 0)]


@pytest.mark.parametrize("int4", [False, True])
@pytest.mark.parametrize("q_scale", [0.25, 1.0])
@pytest.mark.parametrize("g, n, window, sinks", CASES)
def test_the_roundings_pass(g, n, window, sinks, int4, q_scale):
    for seed in range(4):
        r = Rows(g, n, window, sinks, int4, seed, q_scale)
        assert r.worst(r.result()) <= 1.0


@pytest.mark.parametrize("int4", [False, True])
@pytest.mark.parametrize("g, n, window, sinks", CASES)
def test_mistakes_do_not(g, n, window, sinks, int4):
    r = Rows(g, n, window, sinks, int4, 7, 0.25)
    see = paged.visible(n - 1, n, window, sinks)
    tiles = [t for t in range(0, n, 16) if see[t:t + 16].all()]
    wrong = {}
    for name, at in (("first tile", tiles[0]), ("last tile", tiles[-1])):
        s = see.copy()
        s[at:at + 16] = False
        wrong[name] = dict(see=s)
    if n <= 1000:
        s = see.copy()
        s[n - 1] = False
        wrong["newest key"] = dict(see=s)
    if window > 0:
        s = see.copy()
        s[n - 1 - window] = True
        wrong["a key too many"] = dict(see=s)
    if g > 1:
        wrong["another head's query"] = dict(head=0)
    if int4:
        wrong["offset of K"] = dict(k_offset=8.0)
        wrong["offset of V"] = dict(v_offset=8.0)
        wrong["scale of a group"] = dict(k_scale=(1.0, 1.05))
    for name, change in wrong.items():
        assert r.worst(r.result(**change)) > 1.0, name
    flat = r.result()
    flat[..., np.arange(128) != 3] = 0.0
    assert r.worst(flat) > 1.0, "all channels but the one that stands out"
