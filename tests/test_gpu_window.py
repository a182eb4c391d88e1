"""Attention with a sliding window and visible first tokens over BF16 pages and the 4-bit cache, against the oracle."""

import numpy as np
import pytest
import torch

from oracle import paged
from int2_rotated_kv_oscar_gb300 import abi
from int2_rotated_kv_oscar_gb300 import cache as kv
from paged_harness import DEV, attention_error, context, f64, fill_bf16, int4_rows, ints, nan_int4, nan_pages, tables

pytestmark = pytest.mark.gpu


class Case:
    """Requests with queries at p0 .. p0 + count - 1 over a cache of ctx positions; what no query sees is NaN."""

    def __init__(self, Hq, Hkv, spans, window, sinks, int4, seed=0, sm_scale=0.0, give_back=True, q_scale=1.0):
        self.Hq, self.Hkv, self.spans, self.window, self.sinks, self.int4 = Hq, Hkv, spans, window, sinks, int4
        self.sm_scale = sm_scale
        r = np.random.default_rng([seed, Hq, Hkv, len(spans), window + 1, sinks])
        self.n = sum(c for _, c, _ in spans)
        self.ctxs = [c for _, _, c in spans]
        self.table, num_pages = tables(self.ctxs, seed)
        self.ctx = context(Hq, Hkv)
        width = (Hq + 3) * 128  # the queries are part of a wider row
        wide = torch.from_numpy(r.standard_normal((self.n, width)).astype(np.float32) * q_scale).to(DEV, torch.bfloat16)
        self.q = wide[:, 128:128 + Hq * 128].unflatten(1, (Hq, 128))
        self.out = torch.full((self.n, Hq, 128), 9.0, dtype=torch.bfloat16, device=DEV)
        self.pos, self.len = ints([p for p, _, _ in spans]), ints(self.ctxs)
        self.cu = ints(np.concatenate([[0], np.cumsum([c for _, c, _ in spans])]))
        self.single = all(c == 1 for _, c, _ in spans)
        seen = []
        rows = [[], []]
        for p0, count, ctx in spans:
            see = np.zeros(ctx, bool)
            for p in range(p0, p0 + count):
                see |= paged.visible(p, ctx, window, sinks)
            seen.append(see)
            for x in rows:
                y = r.standard_normal((ctx, Hkv, 128)).astype(np.float32)
                y[:, :, 3] *= 20.0
                y[~see] = np.nan
                x.append(torch.from_numpy(y).to(DEV, torch.bfloat16))
        self.held = None
        table = self.table.copy()
        if int4:
            self.pages = nan_int4(num_pages, Hkv)
            self.K, self.V, self.held = [], [], []
            for b, ctx in enumerate(self.ctxs):
                runs = np.flatnonzero(np.diff(np.concatenate([[0], seen[b].astype(int), [0]])))
                for lo, hi in zip(runs[::2], runs[1::2]):
                    abi.oscar_rope_append_int4(
                        self.ctx, kv.int4_view(self.pages, ints(table[b:b + 1])),
                        kv.rope_append_args(rows[0][b][lo:hi], rows[1][b][lo:hi], ints([lo]), cu_seqlens=ints([0, hi - lo]),
                                            max_tokens_per_req=int(hi - lo)))
                if ctx == 0:
                    self.K.append(np.zeros((0, Hkv, 128)))
                    self.V.append(np.zeros((0, Hkv, 128)))
                    self.held.append((np.zeros((0, Hkv)), np.zeros((0, Hkv))))
                    continue
                kc, ks, vc, vs = int4_rows(self.pages, table, b, ctx)
                with np.errstate(invalid="ignore"):
                    self.K.append(paged.levels(kc, ks))
                    self.V.append(paged.levels(vc, vs))
                self.held.append((ks.astype(np.float64).max(-1), vs.astype(np.float64).max(-1)))
            assert abi.oscar_check_device_error(self.ctx) == 0
        else:
            self.k_pages, self.v_pages = nan_pages(num_pages, Hkv)
            for pages, x in ((self.k_pages, rows[0]), (self.v_pages, rows[1])):
                fill_bf16(pages, table, self.ctxs, x)
            self.K, self.V = [f64(x) for x in rows[0]], [f64(x) for x in rows[1]]
        if give_back:  # pages that no query sees are not the request's any more
            for b, see in enumerate(seen):
                for lp in range(table.shape[1]):
                    if not see[64 * lp:64 * lp + 64].any():
                        table[b, lp] = (-1, 1 << 30)[lp % 2]
        self.pt = ints(table)
        _, self.ws, self.ws_bytes = self.workspace = kv.window_workspace(self.ctx)

    def view(self):
        return kv.int4_view(self.pages, self.pt) if self.int4 else kv.bf16_view(self.k_pages, self.v_pages, self.pt)

    def args(self, **kw):
        a = dict(window=self.window, sinks=self.sinks, cu_seqlens=None if self.single else self.cu,
                 max_tokens_per_req=max([c for _, c, _ in self.spans] + [1]), sm_scale=self.sm_scale)
        a.update(kw)
        return kv.window_args(self.q, self.out, self.pos, self.len, max(self.ctxs + [1]), **a)

    def call(self, **kw):
        fn = abi.oscar_window_attention_int4 if self.int4 else abi.oscar_window_attention_bf16
        fn(self.ctx, self.view(), self.args(**kw), self.ws, self.ws_bytes, torch.cuda.current_stream())

    def worst(self):
        pack = self.Hq // self.Hkv <= 4 and (self.single or self.int4)
        return attention_error(f64(self.out), f64(self.q), self.K, self.V, self.spans, self.window, self.sinks, pack,
                               sm_scale=self.sm_scale or 128 ** -0.5, held=self.held)

    def check(self):
        self.call()
        assert abi.oscar_check_device_error(self.ctx) == 0
        assert self.worst() <= 1.0

    def close(self):
        abi.oscar_destroy(self.ctx)


def steps(*lengths):
    return [(n - 1, 1, n) for n in lengths]


SINGLE = [
    dict(Hq=8, Hkv=2, spans=steps(1), window=-1, sinks=0),
    dict(Hq=4, Hkv=1, spans=steps(15, 16, 17, 31, 32, 33, 63, 64, 65), window=-1, sinks=0),
    dict(Hq=8, Hkv=2, spans=steps(1, 2, 16, 17, 64, 100, 129), window=1, sinks=0),
    dict(Hq=8, Hkv=2, spans=steps(1, 5, 70, 500, 1000), window=7, sinks=3),
    dict(Hq=32, Hkv=8, spans=steps(1500, 90, 260), window=200, sinks=64),
    dict(Hq=16, Hkv=2, spans=steps(700, 33, 64), window=65, sinks=70),
    dict(Hq=5, Hkv=1, spans=steps(300, 2), window=0, sinks=5),
    dict(Hq=3, Hkv=3, spans=steps(40, 400), window=16, sinks=16),
    dict(Hq=6, Hkv=1, spans=steps(257), window=-1, sinks=40),
    dict(Hq=8, Hkv=1, spans=steps(5003), window=-1, sinks=0),
    dict(Hq=4, Hkv=1, spans=steps(20011), window=-1, sinks=0),
    dict(Hq=4, Hkv=1, spans=steps(20011), window=9001, sinks=33),
    # nothing to see: an empty cache, no window and no sinks, a query whose window lies beyond what is held
    dict(Hq=8, Hkv=2, spans=[(0, 1, 0), (40, 1, 41), (100, 1, 50)], window=0, sinks=0),
    dict(Hq=8, Hkv=2, spans=[(0, 1, 0), (40, 1, 41), (100, 1, 50), (100, 1, 95)], window=10, sinks=0),
    dict(Hq=2, Hkv=2, spans=[(100, 1, 50), (30, 1, 200)], window=10, sinks=2),
    dict(Hq=8, Hkv=2, spans=steps(130, 77), window=-1, sinks=0, sm_scale=0.5),
]

CHUNKS = [
    dict(Hq=8, Hkv=2, spans=[(0, 5, 5), (60, 9, 69), (7, 0, 7)], window=-1, sinks=0),
    dict(Hq=4, Hkv=1, spans=[(0, 130, 130)], window=-1, sinks=0),
    dict(Hq=4, Hkv=1, spans=[(0, 200, 200), (31, 34, 65)], window=50, sinks=4),
    dict(Hq=8, Hkv=1, spans=[(300, 70, 370), (0, 1, 1)], window=100, sinks=64),
    dict(Hq=2, Hkv=2, spans=[(500, 150, 650)], window=129, sinks=1),
    dict(Hq=5, Hkv=1, spans=[(10, 60, 70)], window=16, sinks=0),
    dict(Hq=3, Hkv=1, spans=[(0, 100, 100)], window=0, sinks=9),
    dict(Hq=4, Hkv=1, spans=[(0, 90, 60), (100, 40, 95)], window=20, sinks=0),  # the last queries see nothing
    dict(Hq=8, Hkv=2, spans=[(1000, 257, 1257)], window=-1, sinks=0),
    dict(Hq=6, Hkv=1, spans=[(130, 65, 195)], window=64, sinks=130),
]


MANY = [  # more work items than the GPU has SMs
    dict(Hq=2, Hkv=1, spans=[((7 * i) % 90, 1 + i % 4, (7 * i) % 90 + 1 + i % 4) for i in range(400)], window=40, sinks=2),
    dict(Hq=64, Hkv=8, spans=[(0, 150, 150), (300, 40, 340), (10, 131, 141), (0, 33, 33), (130, 150, 280)], window=100,
         sinks=4),
    dict(Hq=8, Hkv=8, spans=[(0, 200 + i, 200 + i) for i in range(0, 140, 7)], window=-1, sinks=0),
]


@pytest.mark.parametrize("i", range(len(MANY)))
def test_many_work_items(i):
    c = Case(**MANY[i], int4=False, seed=200 + i)
    c.check()
    first = c.out.clone()
    c.call()
    torch.cuda.synchronize()
    assert torch.equal(first, c.out)
    c.close()


@pytest.mark.parametrize("int4", [False, True])
@pytest.mark.parametrize("i", range(len(SINGLE)))
def test_single_tokens(i, int4):
    c = Case(**SINGLE[i], int4=int4, seed=i)
    c.check()
    c.close()


@pytest.mark.parametrize("int4", [False, True])
@pytest.mark.parametrize("i", range(len(CHUNKS)))
def test_chunks_and_prompts(i, int4):
    c = Case(**CHUNKS[i], int4=int4, seed=100 + i)
    c.check()
    c.close()


@pytest.mark.parametrize("int4", [False, True])
def test_sharp_softmax(int4):
    """Logits in the hundreds: one key takes nearly all the weight, the running maximum moves far."""
    c = Case(8, 2, steps(900, 64, 333), 500, 4, int4, seed=5, q_scale=30.0)
    c.check()
    c.close()


@pytest.mark.parametrize("int4", [False, True])
@pytest.mark.parametrize("spans", [steps(3000, 20), [(2000, 70, 2070)]])
def test_same_result_again_and_on_another_stream_and_captured(spans, int4):
    c = Case(8, 2, spans, 1500, 4, int4, seed=6)
    c.check()
    first = c.out.clone()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        c.out.zero_()
        c.call()
    side.synchronize()
    assert torch.equal(first, c.out)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        c.call()
    c.out.zero_()
    for _ in range(3):
        graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(first, c.out)
    c.close()


def test_aliased_prefix_pages():
    """Two requests that share their first pages see the same rows."""
    c = Case(8, 2, steps(300, 300), -1, 0, False, seed=7)
    c.pt[1, :4] = c.pt[0, :4]
    c.K[1][:256], c.V[1][:256] = c.K[0][:256], c.V[0][:256]
    c.check()
    c.close()


@pytest.mark.parametrize("int4", [False, True])
@pytest.mark.parametrize("spans", [steps(200, 300), [(100, 100, 200), (220, 80, 300)]])
def test_bad_pages_lengths_and_spans(spans, int4):
    c = Case(4, 1, spans, -1, 0, int4, seed=8)
    good = c.pt.clone()
    c.pt[0, 1] = 1 << 20
    c.call()
    assert abi.oscar_check_device_error(c.ctx) == abi.OSCAR_DEVERR_PAGE
    assert torch.isfinite(c.out.float()).all()
    c.pt = good[:, :2].contiguous()
    c.call()
    assert abi.oscar_check_device_error(c.ctx) == abi.OSCAR_DEVERR_LENGTH
    c.pt = good
    c.pos[1] = -2
    c.call()
    assert abi.oscar_check_device_error(c.ctx) == abi.OSCAR_DEVERR_LENGTH
    c.pos[1] = spans[1][0]
    if not c.single:
        n = c.n
        c.out.fill_(9.0)
        c.cu.copy_(ints([0, 100, 90]))
        c.call()
        assert abi.oscar_check_device_error(c.ctx) == abi.OSCAR_DEVERR_TOKENS
        assert (c.out[:100] != 9.0).any() and (c.out[100:] == 9.0).all()
        c.cu.copy_(ints([0, 60, 90]))  # rows 90.. belong to nobody
        c.out.fill_(9.0)
        c.pos[1] = 200
        c.call()
        assert abi.oscar_check_device_error(c.ctx) == 0
        assert (c.out[90:] == 9.0).all()
        c.cu.copy_(ints([0, 100, n]))
        c.pos[1] = spans[1][0]
    c.check()
    c.close()


def test_window_refusals():
    for int4 in (False, True):
        c = Case(8, 2, steps(40), 16, 0, int4)
        fn = abi.oscar_window_attention_int4 if int4 else abi.oscar_window_attention_bf16

        def status(ws=c.ws, size=c.ws_bytes, **change):
            a, v = c.args(), c.view()
            for name, value in change.items():
                setattr(v if hasattr(v, name) and not hasattr(a, name) else a, name, value)
            try:
                fn(c.ctx, v, a, ws, size)
            except abi.OscarError as e:
                return e.status
            return 0

        c.out.fill_(9.0)
        for change in (dict(q=None), dict(out=None), dict(pos=None), dict(ctx_len=None), dict(q=c.q.data_ptr() + 2),
                       dict(out=c.out.data_ptr() + 8), dict(n_tokens=2), dict(n_tokens=-1), dict(max_ctx_len=-1),
                       dict(sinks=-1), dict(sm_scale=float("nan")), dict(sm_scale=float("inf")), dict(q_stride=8 * 128 + 4),
                       dict(q_stride=128), dict(num_pages=0), dict(page_table=None), dict(max_pages_per_req=0),
                       dict(batch=-1)):
            assert status(**change) == 1, change
        assert status(ws=None) == 6 and status(ws=c.ws + 8) == 6 and status(size=c.ws_bytes - 1) == 6
        assert status(batch=0, n_tokens=0) == 0
        assert (c.out == 9.0).all(), "a refused call writes nothing"
        assert abi.oscar_check_device_error(c.ctx) == 0
        c.close()


@pytest.mark.parametrize("int4", [False, True])
def test_prompt_then_decode_steps(int4):
    """As they are used: prompts appended with their positions and attended, then tokens one by one."""
    Hq, Hkv, window, sinks = 8, 2, 60, 4
    prompts, more = [150, 33], 5
    total = [p + more for p in prompts]
    table, num_pages = tables(total, 11)
    ctx = context(Hq, Hkv)
    rope = kv.rope_table(ctx, 512)
    r = np.random.default_rng(12)
    x = [torch.from_numpy(r.standard_normal((t, Hq + 2 * Hkv, 128)).astype(np.float32)).to(DEV, torch.bfloat16) for t in total]
    k_pages, v_pages = nan_pages(num_pages, Hkv)
    pages = nan_int4(num_pages, Hkv)
    pt = ints(table)
    bf16, int4v = kv.bf16_view(k_pages, v_pages, pt), kv.int4_view(pages, pt)
    _, ws, size = kv.window_workspace(ctx)
    append = (abi.oscar_rope_append_int4, int4v) if int4 else (abi.oscar_rope_append_bf16, bf16)
    attend = (abi.oscar_window_attention_int4, int4v) if int4 else (abi.oscar_window_attention_bf16, bf16)
    spans, rows = [(0, p) for p in prompts], [x[b][:p] for b, p in enumerate(prompts)]
    for step in range(more + 1):
        if step:
            spans = [(p + step - 1, 1) for p in prompts]
            rows = [x[b][p + step - 1:p + step] for b, p in enumerate(prompts)]
        qkv = torch.cat(rows)
        q, k, v = qkv[:, :Hq], qkv[:, Hq:Hq + Hkv], qkv[:, Hq + Hkv:]
        q_rot = torch.empty((len(qkv), Hq, 128), dtype=torch.bfloat16, device=DEV)
        out = torch.empty_like(q_rot)
        cu = None if step else ints(np.concatenate([[0], np.cumsum(prompts)]))
        most = 1 if step else max(prompts)
        pos, lens = ints([p for p, _ in spans]), ints([p + c for p, c in spans])
        append[0](ctx, append[1], kv.rope_append_args(k, v, pos, q=q, q_out=q_rot, rope=rope, cu_seqlens=cu,
                                                      max_tokens_per_req=most))
        attend[0](ctx, attend[1], kv.window_args(q_rot, out, pos, lens, max(total), window=window, sinks=sinks,
                                                 cu_seqlens=cu, max_tokens_per_req=most), ws, size)
        assert abi.oscar_check_device_error(ctx) == 0
        K, V, held = [], [], [] if int4 else None
        for b, (p, c) in enumerate(spans):
            n = p + c
            if int4:
                kc, ks, vc, vs = int4_rows(pages, table, b, n)
                K.append(paged.levels(kc, ks))
                V.append(paged.levels(vc, vs))
                held.append((ks.astype(np.float64).max(-1), vs.astype(np.float64).max(-1)))
            else:
                at = torch.arange(n, device=DEV)
                ids = pt[b].long()[at // 64]
                K.append(f64(k_pages[ids, :, at % 64]))
                V.append(f64(v_pages[ids, :, at % 64]))
        got = attention_error(f64(out), f64(q_rot), K, V, [(p, c, p + c) for p, c in spans], window, sinks, False, held=held)
        assert got <= 1.0, step
    abi.oscar_destroy(ctx)


def test_chunk_over_a_prefix_held_in_4_bits():
    """A long prefix in 4 bits is read back into BF16 pages, the chunk is appended there and attends both."""
    Hq, Hkv, prefix, chunk = 8, 2, 200, 40
    table, num_pages = tables([prefix + chunk], 13)
    ctx = context(Hq, Hkv)
    rope = kv.rope_table(ctx, 256)
    r = np.random.default_rng(14)
    x = torch.from_numpy(r.standard_normal((prefix + chunk, Hq + 2 * Hkv, 128)).astype(np.float32)).to(DEV, torch.bfloat16)
    pages, pt = nan_int4(num_pages, Hkv), ints(table)
    k_pages, v_pages = nan_pages(num_pages, Hkv)
    bf16, int4v = kv.bf16_view(k_pages, v_pages, pt), kv.int4_view(pages, pt)
    abi.oscar_rope_append_int4(ctx, int4v, kv.rope_append_args(
        x[:prefix, Hq:Hq + Hkv], x[:prefix, Hq + Hkv:], ints([0]), rope=rope, cu_seqlens=ints([0, prefix]),
        max_tokens_per_req=prefix))
    abi.oscar_int4_to_bf16(ctx, int4v, bf16, ints([0]), ints([prefix]), prefix)
    q_rot = torch.empty((chunk, Hq, 128), dtype=torch.bfloat16, device=DEV)
    out = torch.empty_like(q_rot)
    new = kv.rope_append_args(x[prefix:, Hq:Hq + Hkv], x[prefix:, Hq + Hkv:], ints([prefix]), q=x[prefix:, :Hq], q_out=q_rot,
                              rope=rope, cu_seqlens=ints([0, chunk]), max_tokens_per_req=chunk)
    abi.oscar_rope_append_bf16(ctx, bf16, new)
    abi.oscar_rope_append_int4(ctx, int4v, new)
    _, ws, size = kv.window_workspace(ctx)
    abi.oscar_window_attention_bf16(ctx, bf16, kv.window_args(q_rot, out, ints([prefix]), ints([prefix + chunk]),
                                                              prefix + chunk, cu_seqlens=ints([0, chunk])), ws, size)
    assert abi.oscar_check_device_error(ctx) == 0
    at = torch.arange(prefix + chunk, device=DEV)
    ids = pt[0].long()[at // 64]
    K, V = f64(k_pages[ids, :, at % 64]), f64(v_pages[ids, :, at % 64])
    kc, ks, vc, vs = int4_rows(pages, table, 0, prefix + chunk)
    for rows, codes, scales in ((K, kc, ks), (V, vc, vs)):  # the prefix's rows are what the 4-bit cache stands for
        held = paged.from_rotated(paged.levels(codes, scales))[:prefix]
        assert np.linalg.norm(rows[:prefix] - held) <= 2.0 ** -8 * np.linalg.norm(held)
    assert attention_error(f64(out), f64(q_rot), [K], [V], [(prefix, chunk, prefix + chunk)], -1, 0, False) <= 1.0
    abi.oscar_destroy(ctx)
