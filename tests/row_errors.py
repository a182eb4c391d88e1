"""A check of an attention's rows that a missing key or a wrong constant does not pass: the norm of each row's error
against what the roundings of its operands add up to.

A bound that takes every rounding at its worst, in one direction, grows with the number of keys while the result itself
shrinks; but roundings of different operands are independent.  So, for the result o = sum_j w_j v_j of one query:
  * a weight that is rounded to bf16 is off by at most half a step, 2^-8 of it, evenly: a variance of (2^-8)^2 / 3, and
    sum_j w_j^2 |v_j|^2 of that in o (two bf16 terms: 2^-16); the sum of the weights is taken before the rounding;
  * an error e_j of a logit changes o by w_j e_j (v_j - o).  fp32 sums: 2^-23 for each of the MMA's 8 steps and 16 lanes
    of the sum of their magnitudes, independent from key to key.  4 bits, one fp16 term: the operands h1 = q_(c+2) / 16 and
    h0 = q_c - q_(c+2) / 16, off by at most 2^-11 of themselves, multiply c + 16 c' and c (levels, once the offsets
    cancel) of all keys: each adds the square of its error times the norm of sum_j w_j (its factor)_j (v_j - o);
  * the sums of P V: 2^-23 of the running sum's magnitude a step (truncated, so in one direction);
  * the result's own rounding, 2^-8 of each channel.
The limit takes the independent ones together as six times their standard deviation.
"""

import numpy as np

from oracle import paged


def row_limit(qr, k, v, w, o, sm_scale, g, pack, held, tensor_cores):
    """The limit of one row; k, v [n, 128] as seen, in the cache's basis, w their weights, o the result in that basis."""
    half = 2.0 ** -16 if pack else 2.0 ** -8
    x = float((np.abs(k) @ np.abs(qr)).max())
    ex = (24 * 2.0 ** -23 * x) * sm_scale + 2.0 ** -20
    far = np.abs(v).max()
    n = len(k)
    if held is not None:
        s_k, s_v = held
        ex += 8 * 2.0 ** -23 * 23.5 * s_k * np.abs(qr).sum() * sm_scale
        far = 23.5 * s_v
    d = v - o
    var = (w ** 2 * (half ** 2 / 3 * (v ** 2).sum(1) + (2 * ex) ** 2 * (d ** 2).sum(1))).sum()
    if held is not None and not pack:
        low = np.array([c for c in range(128) if not c & 2])
        m = (k * w[:, None] * sm_scale).T @ d  # [channel][128]: what the result gains with a channel of the query
        h1 = qr[low + 2] / 16
        h0 = qr[low] - h1
        var += (2.0 ** -11) ** 2 / 3 * ((h0 ** 2 * (m[low] ** 2).sum(1)).sum()
                                        + (h1 ** 2 * ((m[low] + 16 * m[low + 2]) ** 2).sum(1)).sum())
    # P V: a warp's share of the keys (eight warps at least share a pair's), or all of them on the tensor cores
    steps = 8 + n / (16 if tensor_cores else 128)
    sums = steps * 2.0 ** -23 * far * np.sqrt(128.0)
    return 2.0 ** -8 * np.linalg.norm(o) + 6 * np.sqrt(var) + sums + 1e-30


def row_errors(out, q, K, V, spans, window, sinks, pack, sm_scale=128 ** -0.5, held=None, tensor_cores=False):
    """The largest |out - o| / limit over the rows of out [n, Hq, 128]; the arguments are attention_error's."""
    worst, i, Hq = 0.0, 0, q.shape[1]
    for b, (p0, count, ctx) in enumerate(spans):
        g = Hq // K[b].shape[1]
        for p in range(p0, p0 + count):
            see = paged.visible(p, ctx, window, sinks)
            for hq in range(Hq):
                if not see.any():
                    assert not out[i, hq].any(), (b, p, hq)
                    continue
                h = hq // g
                k, v = K[b][:ctx, h][see], V[b][:ctx, h][see]
                qr = paged.to_rotated(q[i, hq]) if held is not None else q[i, hq]
                x = k @ qr * sm_scale
                w = np.exp(x - x.max())
                w /= w.sum()
                o = w @ v
                got = paged.to_rotated(out[i, hq]) if held is not None else out[i, hq]
                scales = None if held is None else [float(s[:ctx, h][see].max()) for s in held[b]]
                limit = row_limit(qr, k, v, w, o, sm_scale, g, pack, scales, tensor_cores)
                error = float(np.linalg.norm(got - o))
                assert np.isfinite(error), (b, p, hq)
                worst = max(worst, error / limit)
            i += 1
    return worst
