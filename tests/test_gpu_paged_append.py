"""Position-rotated appends into BF16 pages and the 4-bit cache, and the 4-bit read-back, against the fp64 oracle."""

import ctypes

import numpy as np
import pytest
import torch

from oracle import paged
from int2_rotated_kv_oscar_gb300 import abi
from int2_rotated_kv_oscar_gb300 import cache as kv
from paged_harness import BF16, DEV, context, f64, fill_bf16, int4_rows, ints, nan_int4, nan_pages, rows_of, tables

pytestmark = pytest.mark.gpu

THETA = 1e6


class Case:
    """Requests that append `count` tokens at `pos`, with inputs that are parts of one wider row (or packed)."""

    def __init__(self, Hq, Hkv, spans, rotary=128, interleaved=False, fused=True, seed=0, queries=True, scale=1.0):
        self.Hq, self.Hkv, self.spans, self.rotary, self.interleaved = Hq, Hkv, spans, rotary, interleaved
        r = np.random.default_rng([seed, Hq, Hkv, len(spans)])
        self.n = sum(c for _, c in spans)
        x = r.standard_normal((max(self.n, 1), Hq + 2 * Hkv, 128)).astype(np.float32) * scale
        x[:, :, r.choice(128, 4, replace=False)] *= 20.0
        x = torch.from_numpy(x).to(DEV, torch.bfloat16)[:self.n]
        parts = [x[:, :Hq], x[:, Hq:Hq + Hkv], x[:, Hq + Hkv:]]
        self.q, self.k, self.v = parts if fused else [t.contiguous() for t in parts]
        if not queries:
            self.q = None
        self.q_out = torch.full((self.n, Hq, 128), 7.0, dtype=torch.bfloat16, device=DEV) if queries else None
        self.lengths = [p + c for p, c in spans]
        self.table, self.num_pages = tables(self.lengths, seed)
        self.pos = ints([p for p, _ in spans])
        self.cu = ints(np.concatenate([[0], np.cumsum([c for _, c in spans])]))
        self.most = max([c for _, c in spans] + [1])
        self.ctx = context(Hq, Hkv)
        self.rope = kv.rope_table(self.ctx, max(self.lengths + [1]), rotary, THETA) if rotary else None
        self.pt = ints(self.table)

    def args(self, **kw):
        a = dict(q=self.q, q_out=self.q_out, rope=self.rope, interleaved=self.interleaved, cu_seqlens=self.cu,
                 max_tokens_per_req=self.most)
        if all(c == 1 for _, c in self.spans):
            a["cu_seqlens"] = None
        a.update(kw)
        return kv.rope_append_args(self.k, self.v, self.pos, **a)

    def positions(self):
        return np.concatenate([np.arange(p, p + c) for p, c in self.spans])

    def turned(self, x):
        """fp64 rotation of rows x with the table's own entries, and the magnitudes that the fp32 terms go through."""
        x = f64(x)
        half = self.rotary // 2
        t = f64(self.rope)[self.positions()] if half else np.zeros((len(x), 0))
        c, s = t[:, :half], t[:, half:]
        return paged.rope(x, c, s, self.interleaved), paged.rope(np.abs(x), np.abs(c), -np.abs(s), self.interleaved) + (
            paged.rope(np.abs(x), np.abs(c), np.abs(s), self.interleaved)).clip(min=0) + np.abs(x)

    def close(self):
        abi.oscar_destroy(self.ctx)


CASES = [
    dict(Hq=8, Hkv=2, spans=[(0, 1)]),
    dict(Hq=32, Hkv=8, spans=[(17, 1), (64, 1), (99999, 1), (63, 1)]),
    dict(Hq=5, Hkv=1, spans=[(0, 100)], fused=False),
    dict(Hq=8, Hkv=2, spans=[(0, 37), (61, 6), (5, 0), (128, 64), (15, 1), (33, 95)], rotary=64),
    dict(Hq=4, Hkv=4, spans=[(1000, 130), (3, 5)], interleaved=True),
    dict(Hq=16, Hkv=2, spans=[(7, 41), (48, 16)], rotary=64, interleaved=True),
    dict(Hq=2, Hkv=1, spans=[(16, 16), (0, 15), (31, 2)], rotary=0),
    dict(Hq=24, Hkv=3, spans=[(2, 19)], queries=False),
]


def test_rope_table():
    ctx = context(8, 2)
    for rotary in (64, 128):
        t = f64(kv.rope_table(ctx, 131100, rotary, THETA))
        at = np.array([0, 1, 63, 4097, 99999, 131099])
        a = paged.rope_angles(at, rotary, THETA)
        # half a step of fp32 (entries are at most 1) and the angle's own rounding in fp64
        tol = 2.0 ** -24 + 2.0 ** -50 * a
        assert (np.abs(t[at, :rotary // 2] - np.cos(a)) <= tol).all()
        assert (np.abs(t[at, rotary // 2:] - np.sin(a)) <= tol).all()
    abi.oscar_destroy(ctx)


@pytest.mark.parametrize("i", range(len(CASES)))
def test_append_bf16(i):
    c = Case(**CASES[i], seed=i)
    k_pages, v_pages = nan_pages(c.num_pages, c.Hkv)
    abi.oscar_rope_append_bf16(c.ctx, kv.bf16_view(k_pages, v_pages, c.pt), c.args())
    assert abi.oscar_check_device_error(c.ctx) == 0
    # expected pools: NaN but for the new rows
    want_k, want_v = nan_pages(c.num_pages, c.Hkv)
    at = torch.from_numpy(c.positions()).to(DEV)
    b = torch.from_numpy(np.repeat(np.arange(len(c.spans)), [n for _, n in c.spans])).to(DEV)
    page = c.pt.long()[b, at // 64]
    got = k_pages[page, :, at % 64]
    want_v[page, :, at % 64] = c.v
    assert torch.equal(v_pages.view(torch.int16), want_v.view(torch.int16))
    want_k[page, :, at % 64] = got
    assert torch.equal(k_pages.view(torch.int16), want_k.view(torch.int16)), "only the new rows are written"
    for x, y in ((c.k, got),) + (((c.q, c.q_out),) if c.q is not None else ()):
        want, size = c.turned(x)
        # two products and a sum in fp32 (three roundings of at most 2^-24), then bf16
        assert (np.abs(f64(y) - want) <= BF16 * np.abs(want) + 2.0 ** -22 * size).all()
    c.close()


@pytest.mark.parametrize("i", range(len(CASES)))
def test_append_int4_and_read_back(i):
    c = Case(**CASES[i], seed=i)
    # what the BF16 pages hold is what the 4-bit cache quantises
    k_pages, v_pages = nan_pages(c.num_pages, c.Hkv)
    abi.oscar_rope_append_bf16(c.ctx, kv.bf16_view(k_pages, v_pages, c.pt), c.args())
    q_bf16 = None if c.q_out is None else c.q_out.clone()
    pages = torch.randint(0, 256, (c.num_pages, c.Hkv, abi.INT4_BLOCK_BYTES), dtype=torch.uint8, device=DEV,
                          generator=torch.Generator(DEV).manual_seed(i))
    before = pages.clone()
    view = kv.int4_view(pages, c.pt)
    abi.oscar_rope_append_int4(c.ctx, view, c.args())
    assert abi.oscar_check_device_error(c.ctx) == 0
    if c.q_out is not None:
        assert torch.equal(c.q_out, q_bf16)
    back_k, back_v = nan_pages(c.num_pages, c.Hkv)
    abi.oscar_int4_to_bf16(c.ctx, view, kv.bf16_view(back_k, back_v, c.pt), c.pos, ints([n for _, n in c.spans]), c.most)
    assert abi.oscar_check_device_error(c.ctx) == 0
    compared = excluded = 0
    for b, (p0, count) in enumerate(c.spans):
        n = p0 + count
        if not n:
            continue
        now, was = int4_rows(pages, c.table, b, n), int4_rows(before, c.table, b, n)
        for x, y in zip(now, was):
            assert np.array_equal(x[:p0].view(np.uint8), y[:p0].view(np.uint8)), "older tokens keep their bytes"
        for which, src, back in ((0, k_pages, back_k), (2, v_pages, back_v)):
            x = rows_of(src, c.table, b, n)[p0:]
            xr = paged.to_rotated(x)
            codes, scales = now[which][p0:], now[which + 1][p0:]
            # fp32 sums of 128 exact products (16 terms in an MMA, three additions, one scaling)
            e = 24 * 2.0 ** -23 * np.abs(x).sum(-1, keepdims=True) / np.sqrt(128.0)
            a = np.abs(xr).reshape(xr.shape[:-1] + (2, 64)).max(-1)
            lo, hi = [(np.minimum(a + d, 65504 * 7.5) / 7.5).astype(np.float16) for d in (-e, e)]
            assert ((scales >= lo) & (scales <= hi)).all()
            s = np.repeat(scales.astype(np.float64), 64, axis=-1)
            live = s > 0
            t = np.where(live, xr / np.where(live, s, 1.0) + 8.0, 8.0)
            band = np.where(live, e / np.where(live, s, 1.0), 0.0) + 2.0 ** -19
            near = np.abs(t - np.round(t)) <= band
            want = np.clip(np.floor(t), 0, 15).astype(np.uint8)
            assert ((codes == want) | near).all()
            assert (np.abs(codes.astype(int) - want.astype(int)) <= 1).all()
            compared += int((~near).sum())
            excluded += int(near.sum())
            lev = paged.levels(codes, scales)
            y, held = f64(back[torch.from_numpy(c.table[b][np.arange(p0, n) // 64].astype(np.int64)).to(DEV), :,
                               torch.from_numpy(np.arange(p0, n) % 64).to(DEV)]), paged.from_rotated(lev)
            tol = BF16 * np.abs(held) + 24 * 2.0 ** -23 * np.abs(lev).sum(-1, keepdims=True) / np.sqrt(128.0)
            assert (np.abs(y - held) <= tol).all()
        rest = rows_of(back_k, c.table, b, n)[:p0]
        assert np.isnan(rest).all(), "rows outside the range are left as they were"
    assert excluded <= 1 + 1e-3 * compared
    c.close()


def test_int4_one_at_a_time_equals_a_bulk_append():
    spans = [(3, 50), (30, 5)]
    c = Case(8, 2, spans)
    bulk = nan_int4(c.num_pages, c.Hkv)
    abi.oscar_rope_append_int4(c.ctx, kv.int4_view(bulk, c.pt), c.args())
    single = nan_int4(c.num_pages, c.Hkv)
    start = [0, 50]
    for step in range(50):
        rows = [b for b in range(2) if step < spans[b][1]]
        idx = torch.tensor([start[b] + step for b in rows], device=DEV)
        k, v = c.k[idx], c.v[idx]
        pos = ints([spans[b][0] + step for b in rows])
        view = kv.int4_view(single, c.pt[rows].contiguous())
        abi.oscar_rope_append_int4(c.ctx, view, kv.rope_append_args(k, v, pos, rope=c.rope))
        torch.cuda.synchronize()
    assert torch.equal(bulk, single)
    c.close()


@pytest.mark.parametrize("value", [0.0, 1e-7, 3e-6, 1e5, 3e38])
def test_int4_extreme_rows(value):
    """Groups whose scale is zero, subnormal or above fp16's largest keep the nearest level they have."""
    ctx = context(2, 1)
    x = torch.zeros((16, 1, 128), dtype=torch.bfloat16, device=DEV)
    x[:, 0, 5] = value  # spread by the transform: every rotated channel is +-value / sqrt(128)
    table, n = tables([16], 0)
    pages = nan_int4(n, 1)
    abi.oscar_rope_append_int4(ctx, kv.int4_view(pages, ints(table)),
                               kv.rope_append_args(x, x, ints([0]), cu_seqlens=ints([0, 16]), max_tokens_per_req=16))
    assert abi.oscar_check_device_error(ctx) == 0
    xr = paged.to_rotated(f64(x))
    want, scales, _ = paged.quantise(xr)
    kc, ks, vc, vs = int4_rows(pages, table, 0, 16)
    for codes, s in ((kc, ks), (vc, vs)):
        assert np.array_equal(s, scales)
        assert np.array_equal(codes, want)
    abi.oscar_destroy(ctx)


def test_queries_may_turn_in_place():
    c = Case(8, 2, [(9, 33)])
    apart = c.args()
    k_pages, v_pages = nan_pages(c.num_pages, c.Hkv)
    view = kv.bf16_view(k_pages, v_pages, c.pt)
    abi.oscar_rope_append_bf16(c.ctx, view, apart)
    abi.oscar_rope_append_bf16(c.ctx, view, c.args(q_out=c.q))
    torch.cuda.synchronize()
    assert torch.equal(c.q, c.q_out)
    c.close()


def test_rows_of_no_request_and_bad_spans():
    c = Case(8, 2, [(0, 10), (4, 20), (2, 5)])
    bad = ints([0, 10, 8, 35])  # the second request's tokens run backwards, the third owns more than declared
    k_pages, v_pages = nan_pages(c.num_pages, c.Hkv)
    pages = nan_int4(c.num_pages, c.Hkv)
    for call, view in ((abi.oscar_rope_append_bf16, kv.bf16_view(k_pages, v_pages, c.pt)),
                       (abi.oscar_rope_append_int4, kv.int4_view(pages, c.pt))):
        c.q_out.fill_(7.0)
        call(c.ctx, view, c.args(cu_seqlens=bad))
        assert abi.oscar_check_device_error(c.ctx) == abi.OSCAR_DEVERR_TOKENS
        assert (c.q_out[:10] != 7.0).any() and (c.q_out[10:] == 7.0).all()
        c.q_out.fill_(7.0)
        call(c.ctx, view, c.args(cu_seqlens=ints([0, 10, 20, 20])))  # rows 20.. belong to nobody
        assert abi.oscar_check_device_error(c.ctx) == 0
        assert (c.q_out[20:] == 7.0).all()
    c.close()


def test_bad_pages_and_positions_set_error_bits():
    c = Case(8, 2, [(0, 70)])
    k_pages, v_pages = nan_pages(c.num_pages, c.Hkv)
    pages = nan_int4(c.num_pages, c.Hkv)
    table = c.table.copy()
    table[0, 1] = c.num_pages  # one past the pool
    bf16, int4 = (lambda t: kv.bf16_view(k_pages, v_pages, ints(t))), (lambda t: kv.int4_view(pages, ints(t)))
    for call, view in ((abi.oscar_rope_append_bf16, bf16), (abi.oscar_rope_append_int4, int4)):
        call(c.ctx, view(table), c.args())
        assert abi.oscar_check_device_error(c.ctx) == abi.OSCAR_DEVERR_PAGE
        call(c.ctx, view(table[:, :1]), c.args())  # positions 64.. have no entry
        assert abi.oscar_check_device_error(c.ctx) == abi.OSCAR_DEVERR_LENGTH
        call(c.ctx, view(c.table), c.args(rope=c.rope[:60].contiguous()))  # nor a row in the rope table
        assert abi.oscar_check_device_error(c.ctx) == abi.OSCAR_DEVERR_LENGTH
        for first in (-3, 2 ** 31 - 40):
            c.pos.fill_(first)
            call(c.ctx, view(c.table), c.args())
            assert abi.oscar_check_device_error(c.ctx) == abi.OSCAR_DEVERR_LENGTH
        c.pos.fill_(0)
        call(c.ctx, view(c.table), c.args())
        assert abi.oscar_check_device_error(c.ctx) == 0
    one = ints([0])
    for start, count, most, t4, tb, want in ((0, 70, 70, table, c.table, abi.OSCAR_DEVERR_PAGE),
                                             (0, 70, 70, c.table, table, abi.OSCAR_DEVERR_PAGE),
                                             (0, 70, 70, c.table[:, :1], c.table, abi.OSCAR_DEVERR_LENGTH),
                                             (-1, 70, 70, c.table, c.table, abi.OSCAR_DEVERR_LENGTH),
                                             (0, 70, 69, c.table, c.table, abi.OSCAR_DEVERR_TOKENS),
                                             (0, -5, 69, c.table, c.table, 0), (0, 70, 70, c.table, c.table, 0)):
        abi.oscar_int4_to_bf16(c.ctx, int4(t4), bf16(tb), one + start, one + count, most)
        assert abi.oscar_check_device_error(c.ctx) == want
    c.close()


def test_append_refusals():
    c = Case(8, 2, [(0, 16)])
    k_pages, v_pages = nan_pages(c.num_pages, c.Hkv)
    pages = nan_int4(c.num_pages, c.Hkv)
    views = ((abi.oscar_rope_append_bf16, kv.bf16_view(k_pages, v_pages, c.pt)),
             (abi.oscar_rope_append_int4, kv.int4_view(pages, c.pt)))

    def status(call, view, **change):
        a = c.args()
        for name, value in change.items():
            setattr(a, name, value)
        with pytest.raises(abi.OscarError) as e:
            call(c.ctx, view, a)
        return e.value.status

    for call, view in views:
        for change in (dict(k=None), dict(v=None), dict(pos=None), dict(q_out=None), dict(q=None), dict(rope=None),
                       dict(k=c.k.data_ptr() + 2), dict(q_out=c.q_out.data_ptr() + 8),
                       dict(k_stride=2 * 128 + 4), dict(v_stride=128), dict(q_stride=-8), dict(q_out_stride=8),
                       dict(rotary_dim=-64), dict(rotary_dim=130), dict(interleaved=2), dict(n_tokens=-1),
                       dict(rope_positions=0), dict(max_tokens_per_req=0), dict(cu_seqlens=None)):
            assert status(call, view, **change) == 1, change
        for rotary in (32, 96, 126):
            assert status(call, view, rotary_dim=rotary) == 2
        for field, value in (("num_pages", 0), ("page_table", None), ("max_pages_per_req", 0), ("batch", -1)):
            old = getattr(view, field)
            setattr(view, field, value)
            assert status(call, view) == 1, field
            setattr(view, field, old)
        view.batch = 0
        call(c.ctx, view, c.args())  # no requests: nothing to do
        view.batch = 1
        a = c.args()
        a.n_tokens = 0
        call(c.ctx, view, a)
    lib = abi.load()
    one = ints([0])
    v4, vb = views[1][1], views[0][1]
    ref = ctypes.byref
    assert lib.oscar_int4_to_bf16(c.ctx, ref(v4), ref(vb), None, one.data_ptr(), 1, None) == 1
    assert lib.oscar_int4_to_bf16(c.ctx, ref(v4), ref(vb), one.data_ptr(), one.data_ptr(), -1, None) == 1
    assert lib.oscar_int4_to_bf16(c.ctx, None, ref(vb), one.data_ptr(), one.data_ptr(), 1, None) == 1
    t = torch.zeros((4, 128), device=DEV)
    for args, want in (((t.data_ptr(), 4, 96, 1e4), 2), ((t.data_ptr(), 4, 0, 1e4), 1), ((t.data_ptr(), 4, 128, 0.0), 1),
                       ((t.data_ptr(), -1, 128, 1e4), 1), ((None, 4, 128, 1e4), 1),
                       ((t.data_ptr(), 4, 128, float("nan")), 1), ((t.data_ptr(), 0, 128, 1e4), 0)):
        assert lib.oscar_rope_table(c.ctx, *args, None) == want
    assert torch.isnan(k_pages).all() and (pages == 0xFF).all(), "a refused call writes nothing"
    with pytest.raises(ValueError):
        kv.rope_append_args(c.k[:, :, :64], c.v, c.pos)
    c.close()


def test_rotated_rows_feed_the_mixed_cache_at_once():
    """q_out as the K of the mixed cache's append of a fresh prompt, which copies BF16 rows beside the kernel before it."""
    H, n = 2, 6000
    ctx = context(H, H)
    eye = np.eye(128, dtype=np.float32)
    abi.oscar_load_rotation(ctx, 0, eye, eye, 1.0, 1.0)
    mixed = kv.MixedCache(1, H, n // 64 + 2, 1, 1, 1, n // 64 + 2)
    mixed.page_table.copy_(torch.arange(n // 64 + 2, device=DEV, dtype=torch.int32)[None])
    rope = kv.rope_table(ctx, n)
    k_pages, v_pages = nan_pages(n // 64 + 1, H)
    view = kv.bf16_view(k_pages, v_pages, torch.arange(n // 64 + 1, device=DEV, dtype=torch.int32)[None])
    pages = nan_int4(n // 64 + 1, H)
    view4 = kv.int4_view(pages, torch.arange(n // 64 + 1, device=DEV, dtype=torch.int32)[None])
    pos, cu = ints([0]), ints([0, n])
    for i in range(6):
        x = torch.randn(n, 2 * H, 128, generator=torch.Generator(DEV).manual_seed(i), device=DEV).to(torch.bfloat16)
        turned = torch.full((n, H, 128), float("nan"), dtype=torch.bfloat16, device=DEV)
        rows = kv.rope_append_args(x[:, :H], x[:, H:], pos, q=x[:, :H], q_out=turned, rope=rope, cu_seqlens=cu)
        values = x[:, H:].contiguous()
        torch.cuda.synchronize()
        if i % 2:
            abi.oscar_rope_append_int4(ctx, view4, rows)
        else:
            abi.oscar_rope_append_bf16(ctx, view, rows)
        abi.oscar_kv_append(ctx, 0, mixed.view(0), kv.append_args(turned, values, pos, cu_seqlens=cu, fresh_ring=True))
        assert abi.oscar_check_device_error(ctx) == 0
        at = torch.arange(n - 256, n, device=DEV)
        assert torch.equal(mixed.k_ring[0][0][:, (at - 64) % 256].transpose(0, 1), turned[at])
        assert torch.equal(mixed.k_sink[0][0].transpose(0, 1), turned[:64])
    abi.oscar_destroy(ctx)
