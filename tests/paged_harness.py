"""Shared setup for the GPU tests of the one-kind paged caches: contexts, pools full of NaN, oracle comparisons.

Tolerances: a rounding to bf16 is off by at most half a step, 2^-8 of the value; sums of fp32 terms by at most one step
(2^-23, the tensor cores truncate) of the sum of their magnitudes for each addition.
"""

import numpy as np
import torch

from oracle import paged
from int2_rotated_kv_oscar_gb300 import abi
from int2_rotated_kv_oscar_gb300 import cache as kv

BF16 = 2.0 ** -8
DEV = "cuda"


def context(Hq, Hkv):
    return abi.oscar_create(abi.oscar_config(num_layers=1, num_q_heads=Hq, num_kv_heads=Hkv, head_dim=128, page_size=64,
                                             sink=64, recent=256, group=64, device=0))


def ints(x):
    return torch.from_numpy(np.ascontiguousarray(x, dtype=np.int32)).to(DEV)


def f64(t):
    return t.detach().float().cpu().numpy().astype(np.float64)


def tables(lengths, seed, extra=2):
    """A shuffled page table [batch, max_pages] for requests of these lengths (-1 beyond them) and the pool's size."""
    need = [-(-int(n) // 64) for n in lengths]
    perm = np.random.default_rng(seed).permutation(sum(need) + extra)
    table = np.full((len(need), max(max(need), 1)), -1, np.int32)
    at = 0
    for b, n in enumerate(need):
        table[b, :n] = perm[at:at + n]
        at += n
    return table, sum(need) + extra


def nan_pages(num_pages, Hkv):
    return [torch.full((num_pages, Hkv, 64, 128), float("nan"), dtype=torch.bfloat16, device=DEV) for _ in range(2)]


def nan_int4(num_pages, Hkv):
    """Pages nobody wrote: every code 15, every scale a NaN."""
    return torch.full((num_pages, Hkv, abi.INT4_BLOCK_BYTES), 0xFF, dtype=torch.uint8, device=DEV)


def fill_bf16(pages, table, lengths, rows):
    """rows[b] [n, Hkv, 128] (torch) into the pages at positions 0..n-1."""
    for b, n in enumerate(lengths):
        if n:
            at = torch.arange(int(n), device=DEV)
            ids = torch.from_numpy(table[b].astype(np.int64)).to(DEV)[at // 64]
            pages[ids, :, at % 64] = rows[b].to(DEV, torch.bfloat16)


def rows_of(pages, table, b, n):
    """fp64 [n, Hkv, 128] of request b's positions 0..n-1."""
    at = np.arange(n)
    ids = torch.from_numpy(table[b][at // 64].astype(np.int64)).to(DEV)
    return f64(pages[ids, :, torch.from_numpy(at % 64).to(DEV)])


def int4_rows(pages, table, b, n):
    """Codes and scales of request b's positions 0..n-1: kc [n, Hkv, 128], ks [n, Hkv, 2], vc, vs."""
    host = pages.cpu().numpy()
    out = [[], [], [], []]
    for lp in range(-(-n // 64)):
        parts = [paged.unpack_block(host[table[b, lp], h]) for h in range(host.shape[1])]
        for i in range(4):
            out[i].append(np.stack([p[i] for p in parts], axis=1))
    return [np.concatenate(o)[:n] if o else None for o in out]


def attention_error(out, q, K, V, spans, window, sinks, pack, sm_scale=128 ** -0.5, held=None):
    """Compare out [n, Hq, 128] with the oracle for every query row; returns the largest |difference| / tolerance.

    K, V: per request [n, Hkv, 128] fp64 in the cache's basis; spans: (first position, count, ctx_len) per request.
    pack: the weights enter their products as two bf16 terms (2^-16) instead of one (2^-8).
    held: 4-bit caches: per request (s_k, s_v) [n, Hkv], the largest scale of each row; then K and V are in the rotated
    basis, the query goes in as fp16 (half a step: 2^-11 of a channel; with pack a second term takes it below 2^-16) and
    two channels' codes are one operand, c + 16 c': q' / 16, whose rounding reaches c and 16 c', and q - q' / 16, whose
    rounding reaches c: with levels of at most 7.5 scales |q'| 7.5 / 8 more than each channel's own part.  The levels' 7.5
    cancels in fp32 against the codes: terms of at most 15 + 15 / 16 + 7.5 scales.
    """
    worst, i = 0.0, 0
    Hq = q.shape[1]
    for b, (p0, count, ctx) in enumerate(spans):
        g = Hq // K[b].shape[1]
        for p in range(p0, p0 + count):
            for hq in range(Hq):
                h = hq // g
                k, v = K[b][:ctx, h], V[b][:ctx, h]
                qv = q[i, hq]
                qr = paged.to_rotated(qv) if held is not None else qv
                o, A, X = paged.attend(qr, k, v, p, window, sinks, sm_scale)
                # the logits: 128 fp32 additions; the weights' error is its exponential's, in numerator and sum
                ex = 128 * 2.0 ** -23 * X * sm_scale + 2.0 ** -21
                w = 2.0 ** -15 if pack else BF16
                if held is not None:
                    see = paged.visible(p, len(k), window, sinks)
                    sk, sv = (float(s[:ctx, h][see].max()) if see.any() else 0.0 for s in held[b])
                    r = 2.0 ** -16 if pack else 2.0 ** -11
                    ex += (r * X + (r * 7.5 / 8 + 8 * 2.0 ** -23 * 23.5) * sk * np.abs(qr).sum()) * sm_scale
                    steps = len(k) / 16 + 8
                    d = (w + 2 * ex) * A + (2.0 ** -16 + steps * 2.0 ** -23) * 23.5 * sv
                    o, slack = paged.from_rotated(o), np.full(128, d.sum() / np.sqrt(128.0))
                else:
                    slack = (w + 2 * ex + (len(k) / 16) * 2.0 ** -23) * A
                tol = BF16 * np.abs(o) + slack + 1e-30
                diff = np.abs(out[i, hq] - o)
                assert np.isfinite(diff).all(), (b, p, hq)
                worst = max(worst, float((diff / tol).max()))
            i += 1
    return worst
