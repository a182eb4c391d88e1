"""Cases and plain forms of the paged-cache operators: the append of keys and values with the position rotation
(into BF16 pages and into a cache held in 4 bits), the read-back of the 4-bit cache into BF16 pages, and the
attention with a sliding window and visible first tokens over either cache.

``listed()`` and ``draw()`` name cases, ``prepare()`` makes a case's inputs on the GPU, ``run()`` makes one pass:
with ``own`` the framework's calls, otherwise the same operators in elementary torch operations.  ``exact()`` is
the operator's definition in 64 bits.
"""

import math

import numpy as np
import torch

own = False

D = 128            # channels of a head
PAGE = 64          # tokens of a page
TILE = 16          # tokens of a 4-bit tile
TILE_BYTES = 2176  # K codes 1024 | V codes 1024 | K scales 64 | V scales 64
BLOCK = 4 * TILE_BYTES
THETA = 1.0e6

# ---------------------------------------------------------------- cases


def listed():
    return [
        # one decode step's new token of 64 requests of 8K-128K tokens, from a fused QKV projection
        dict(name="append_bf16_step", op="append_bf16", hq=32, hkv=8, batch=64, tokens=1, lo=8192, hi=131072, rotary=128,
             interleaved=False, fused=True),
        # four prompts of uneven length prefilled together; half of the channels rotated, as adjacent pairs
        dict(name="append_bf16_prompts", op="append_bf16", hq=64, hkv=8, batch=4, tokens=8192, lo=0, hi=0, rotary=64,
             interleaved=True, fused=True),
        # the serving batch's decode step into the 4-bit cache, and the rows it now holds
        dict(name="append_int4_step", op="append_int4", hq=32, hkv=8, batch=28, tokens=1, lo=100000, hi=100000, rotary=128,
             interleaved=False, fused=True),
        # a long prompt's K and V (131,072 tokens x 8 heads) into the 4-bit cache, and read back
        dict(name="append_int4_prompt", op="append_int4", hq=0, hkv=8, batch=1, tokens=131072, lo=0, hi=0, rotary=128,
             interleaved=False, fused=False),
        # a chunk's prefix taken out of the 4-bit cache into BF16 pages for the chunk's attention
        dict(name="read_int4_100k", op="read_int4", hq=32, hkv=8, batch=1, lo=99991, hi=99991),
        # batch-1 decode at a 100,000-token context over the 4-bit cache
        dict(name="attend_int4_100k", op="attend_int4", hq=32, hkv=8, batch=1, tokens=1, lo=100000, hi=100000, window=-1,
             sinks=0),
        # ragged requests of 8K-128K tokens, eight query heads to a KV head
        dict(name="attend_int4_ragged", op="attend_int4", hq=64, hkv=8, batch=8, tokens=1, lo=8192, hi=131072, window=-1,
             sinks=0),
        # a windowed layer of the 28-request batch over the 4-bit cache
        dict(name="attend_int4_window", op="attend_int4", hq=32, hkv=8, batch=28, tokens=1, lo=90000, hi=100000,
             window=4096, sinks=64),
        # the smallest call: one short request of a small model
        dict(name="attend_bf16_small", op="attend_bf16", hq=8, hkv=2, batch=1, tokens=1, lo=4096, hi=4096, window=256,
             sinks=64),
        # a windowed layer of 64 decoding requests
        dict(name="attend_bf16_step", op="attend_bf16", hq=32, hkv=8, batch=64, tokens=1, lo=8192, hi=131072, window=4096,
             sinks=4),
        # a 256-token chunk at the end of a 100,000-token context that it sees whole
        dict(name="attend_bf16_chunk", op="attend_bf16", hq=32, hkv=8, batch=1, tokens=256, lo=100000, hi=100000,
             window=-1, sinks=0),
        # three prompts of uneven length through a windowed layer with four sinks
        dict(name="attend_bf16_prompts", op="attend_bf16", hq=32, hkv=8, batch=3, tokens=12288, lo=0, hi=0, window=4096,
             sinks=4),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["append_bf16", "append_int4", "read_int4", "attend_int4", "attend_int4", "attend_bf16", "attend_bf16"])
    hkv = rng.choice([1, 2, 4, 8])
    hq = hkv * rng.choice([1, 2, 4, 5, 8])
    if op == "read_int4":
        batch = _log(rng, 1, 16)
        hi = _log(rng, 1, 100000 // batch)
        return dict(op=op, hq=hq, hkv=hkv, batch=batch, lo=max(1, hi // 3), hi=hi)
    step = rng.random() < 0.5
    if op.startswith("append"):
        batch = _log(rng, 1, 64) if step else _log(rng, 1, 6)
        tokens = 1 if step else _log(rng, 2, 32768 // batch)
        hi = _log(rng, 1, 131072) if step or rng.random() < 0.5 else 0
        rotary = rng.choice([0, 64, 128, 128])
        return dict(op=op, hq=hq, hkv=hkv, batch=batch, tokens=tokens, lo=hi // 2, hi=hi, rotary=rotary,
                    interleaved=rng.random() < 0.4, fused=rng.random() < 0.5)
    if op == "attend_int4" or step:
        batch = _log(rng, 1, 64)
        hi = _log(rng, 1, 131072)
        hi = max(1, min(hi, 700000 // batch))
        window = -1 if rng.random() < 0.4 else _log(rng, 1, 8192)
        # a windowed layer's sinks, or none
        sinks = rng.choice([0, 1, 4, 64, rng.randint(1, 200)]) if window >= 0 else 0
        return dict(op=op, hq=hq, hkv=hkv, batch=batch, tokens=1, lo=max(1, hi // 4), hi=hi, window=window, sinks=sinks)
    batch = _log(rng, 1, 4)
    tokens = _log(rng, 2, 8192 // batch)
    hi = _log(rng, tokens, tokens + 8192) if rng.random() < 0.6 else 0
    window = -1 if rng.random() < 0.3 else _log(rng, 1, 4096)
    sinks = rng.choice([0, 4, 64, rng.randint(1, 200)]) if window >= 0 else 0
    return dict(op=op, hq=hq, hkv=hkv, batch=batch, tokens=tokens, lo=hi, hi=hi, window=window, sinks=sinks)


def _spans(case):
    """(first position, number of new tokens, length) of each request, on the host: the case's own, whatever the seed."""
    n = case["batch"]
    r = np.random.RandomState(n + case["hi"])
    length = r.randint(case["lo"], case["hi"] + 1, n).astype(np.int64)
    if n > 1:
        length[r.randint(n)] = case["hi"]
    t = case.get("tokens", 0)
    count = np.full(n, t, np.int64)
    if t > 1 and n > 1:
        count = r.randint(max(1, t // 2), t + 1, n).astype(np.int64)
        count[r.randint(n)] = t
    if case["op"] == "read_int4":
        return np.zeros_like(length), count, length
    if case["op"].startswith("append") or length.max() == 0:
        return length, count, length + count  # the new tokens come after `length` cached ones
    length = np.maximum(length, count)
    return length - count, count, length      # the queries are the last `count` of the cached ones


def _visible_pages(case, first, count, length):
    """A truth value for each logical page of a request: whether the operator may touch it."""
    pages = int(-(-length.max() // PAGE))
    at = np.arange(pages)[None, :] * PAGE
    end = length[:, None]
    if case["op"].startswith("append"):
        return (at + PAGE > first[:, None]) & (at < end)
    if case["op"] == "read_int4":
        return at < end
    low = first[:, None] - case["window"] + 1 if case["window"] >= 0 else np.zeros_like(end)
    return ((at + PAGE > low) | (at < case["sinks"])) & (at < end)


def prepare(case, seed):
    first, count, length = _spans(case)
    seen = _visible_pages(case, first, count, length)
    hq, hkv, batch = case["hq"], case["hkv"], case["batch"]
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    dev = torch.device("cuda")
    n_pages = int(seen.sum()) + 1
    order = np.random.RandomState((seed + 1) % (1 << 31)).permutation(n_pages)[: n_pages - 1]
    table = np.full(seen.shape, -1, np.int32)  # pages that left the window have been given back
    table[seen] = order
    ints = lambda x: torch.from_numpy(np.ascontiguousarray(x, dtype=np.int32)).to(dev)  # noqa: E731
    s = dict(case=case, n=int(count.sum()), most=int(max(1, count.max())), longest=int(length.max()), pos=ints(first),
             cu=ints(np.concatenate([[0], np.cumsum(count)])), count=ints(count), length=ints(length), table=ints(table))

    def outliers(x):
        """Four channels of each head stand out by a factor of 20."""
        r = np.random.RandomState((seed + 2) % (1 << 31))
        scale = torch.ones(x.shape[-2:])
        for h in range(x.shape[-2]):
            scale[h, torch.from_numpy(r.choice(D, 4, replace=False))] = 20.0
        return x.mul_(scale.to(dev))

    def randn(*shape):
        return torch.randn(shape, generator=g, device=dev)

    n = s["n"]
    if case["op"].startswith("append"):
        heads = [hq, hkv, hkv]
        x = [randn(n, h, D) for h in heads]
        x = [outliers(t) if t.shape[1] and i else t for i, t in enumerate(x)]
        x = [t.to(torch.bfloat16).reshape(n, -1) for t in x]
        if case["fused"]:  # views of one projection's output
            x = list(torch.cat(x, 1).split([h * D for h in heads], 1))
        s["q"], s["k"], s["v"] = [t.unflatten(1, (h, D)) if h else None for t, h in zip(x, heads)]
        s["q_out"] = torch.zeros((n, hq, D), dtype=torch.bfloat16, device=dev) if hq else None
        positions = s["longest"]
        half = case["rotary"] // 2
        if half:
            angle = torch.arange(positions, dtype=torch.float64, device=dev)[:, None] * (
                THETA ** (-torch.arange(half, dtype=torch.float64, device=dev) / half))[None, :]
            s["rope"] = torch.cat([angle.cos(), angle.sin()], 1).to(torch.float32)
        else:
            s["rope"] = None
    if case["op"].startswith("attend"):
        s["q"] = randn(n, hq, D).to(torch.bfloat16)
        s["out"] = torch.zeros((n, hq, D), dtype=torch.bfloat16, device=dev)
    if "int4" in case["op"]:
        if case["op"] == "append_int4":
            s["pages"] = torch.zeros((n_pages, hkv, BLOCK), dtype=torch.uint8, device=dev)
        else:
            shape = (n_pages, hkv, BLOCK // TILE_BYTES, TILE_BYTES)
            a, b = [torch.randint(0, 256, shape, dtype=torch.uint8, device=dev, generator=g) for _ in range(2)]
            low, high = ((a & 15) + (b & 15)) >> 1, ((a >> 4) + (b >> 4) + 1) >> 1
            pages = low | (high << 4)
            scale = (randn(*shape[:3], 64).mul_(0.25).exp_().mul_(0.3)).to(torch.float16)
            pages[..., 2048:] = scale.view(torch.uint8)
            s["pages"] = pages.view(n_pages, hkv, BLOCK)
    if case["op"] in ("append_int4", "read_int4"):  # the BF16 pages that the rows are read back into
        s["k_pages"], s["v_pages"] = [torch.zeros((n_pages, hkv, PAGE, D), dtype=torch.bfloat16, device=dev) for _ in range(2)]
    elif case["op"] == "append_bf16":
        s["k_pages"], s["v_pages"] = [torch.zeros((n_pages, hkv, PAGE, D), dtype=torch.bfloat16, device=dev) for _ in range(2)]
    elif case["op"] == "attend_bf16":
        s["k_pages"], s["v_pages"] = [
            outliers(randn(n_pages, PAGE, hkv, D)).to(torch.bfloat16).transpose(1, 2).contiguous() for _ in range(2)]
    return s


# ---------------------------------------------------------------- the framework's calls

_contexts = {}  # one library handle for each head shape, as a user's program keeps it


def _plan(s):
    """The views, argument blocks and workspace that a user's program makes once for its tensors."""
    from int2_rotated_kv_oscar_gb300 import abi
    from int2_rotated_kv_oscar_gb300 import cache as kv
    c = s["case"]
    heads = (c["hq"] or c["hkv"], c["hkv"])
    if heads not in _contexts:
        _contexts[heads] = abi.oscar_create(abi.oscar_config(
            num_layers=1, num_q_heads=heads[0], num_kv_heads=heads[1], head_dim=D, page_size=PAGE, sink=64, recent=256,
            group=64, device=torch.cuda.current_device()))
    p = dict(ctx=_contexts[heads], abi=abi)
    if "int4" in c["op"]:
        p["int4"] = kv.int4_view(s["pages"], s["table"])
    if "k_pages" in s:
        p["bf16"] = kv.bf16_view(s["k_pages"], s["v_pages"], s["table"])
    if c["op"].startswith("append"):
        p["args"] = kv.rope_append_args(s["k"], s["v"], s["pos"], q=s["q"], q_out=s["q_out"], rope=s["rope"],
                                        interleaved=c["interleaved"], cu_seqlens=s["cu"] if s["most"] > 1 else None,
                                        max_tokens_per_req=s["most"])
    elif c["op"].startswith("attend"):
        p["args"] = kv.window_args(s["q"], s["out"], s["pos"], s["length"], s["longest"], window=c["window"],
                                   sinks=c["sinks"], cu_seqlens=s["cu"] if s["most"] > 1 else None,
                                   max_tokens_per_req=s["most"])
        p["workspace"] = kv.window_workspace(p["ctx"])
    return p


def _own(s):
    p = s.get("plan")
    if p is None:
        p = s["plan"] = _plan(s)
    abi, ctx, op = p["abi"], p["ctx"], s["case"]["op"]
    stream = torch.cuda.current_stream()
    if op == "append_bf16":
        abi.oscar_rope_append_bf16(ctx, p["bf16"], p["args"], stream)
        return dict(q=s["q_out"], k=s["k_pages"], v=s["v_pages"])
    if op == "append_int4":
        abi.oscar_rope_append_int4(ctx, p["int4"], p["args"], stream)
        abi.oscar_int4_to_bf16(ctx, p["int4"], p["bf16"], s["pos"], s["count"], s["most"], stream)
        return dict(q=s["q_out"], k=s["k_pages"], v=s["v_pages"])
    if op == "read_int4":
        abi.oscar_int4_to_bf16(ctx, p["int4"], p["bf16"], s["pos"], s["length"], s["longest"], stream)
        return dict(q=None, k=s["k_pages"], v=s["v_pages"])
    attend = abi.oscar_window_attention_int4 if op == "attend_int4" else abi.oscar_window_attention_bf16
    _, pointer, size = p["workspace"]
    attend(ctx, p["int4" if op == "attend_int4" else "bf16"], p["args"], pointer, size, stream)
    return dict(out=s["out"])


# ---------------------------------------------------------------- the plain forms


def _hadamard(x):
    """x H / sqrt(128) along the last axis, H_ij = (-1)^popcount(i & j)."""
    i = torch.arange(D, device=x.device)
    odd = i[:, None] & i[None, :]
    odd = odd ^ (odd >> 4)
    odd = odd ^ (odd >> 2)
    odd = (odd ^ (odd >> 1)) & 1
    return (x @ (1 - 2 * odd).to(x.dtype)) * (1.0 / math.sqrt(D))


def _nibbles(dev):
    """Where rotated channel j of a token has its nibble: (K byte in the token's 64, K shift, V lane part, V word, V shift)."""
    j = torch.arange(D, device=dev)
    kn = 4 * (j & 1) + 2 * ((j >> 2) & 1) + ((j >> 1) & 1)
    k_byte = 16 * ((j >> 3) & 3) + 4 * (j >> 5) + (kn >> 1)
    v_lane = 4 * ((j & 3) + 4 * ((j >> 3) & 1))
    v_word = ((j >> 2) & 1) + 2 * (j >> 5)
    return k_byte, 4 * (kn & 1), v_lane, v_word, 4 * ((j >> 4) & 1)


def _places(s, t):
    """Byte offsets in a block of the codes of tokens t (0..63): K and V [len(t), 128], and of their scales [len(t), 2]."""
    k_byte, k_shift, v_lane, v_word, v_shift = _nibbles(t.device)
    tile, u = (t >> 4) * TILE_BYTES, t & 15
    k = (tile + 64 * u)[..., None] + k_byte
    v = (tile + 1024)[..., None] + 512 * (v_word >> 2) + 16 * (v_lane + ((u & 7) >> 1)[..., None]) + 4 * (v_word & 3) + (
        2 * (u & 1) + (u >> 3))[..., None]
    pair = torch.arange(2, device=t.device)
    ks = (tile + 2048 + 4 * u)[..., None] + 2 * pair
    return k, k_shift, v, v_shift, ks, ks + 64


def _rows(s):
    """(request, position) of every new token."""
    i = torch.arange(s["n"], device=s["cu"].device)
    b = (torch.searchsorted(s["cu"].long(), i, right=True) - 1).clamp(0, s["case"]["batch"] - 1)
    return b, s["pos"].long()[b] + i - s["cu"].long()[b]


def _rope(x, s, at, dtype):
    """The position rotation of rows x [n, heads, 128] at positions `at`."""
    rotary = s["case"]["rotary"]
    x = x.to(dtype)
    if not rotary:
        return x
    half = rotary // 2
    cos, sin = s["rope"].to(dtype)[at][:, None, :half], s["rope"].to(dtype)[at][:, None, half:]
    if s["case"]["interleaved"]:
        a, b = x[..., 0:rotary:2], x[..., 1:rotary:2]
        y = torch.stack([a * cos - b * sin, b * cos + a * sin], -1).flatten(-2)
    else:
        a, b = x[..., :half], x[..., half:rotary]
        y = torch.cat([a * cos - b * sin, b * cos + a * sin], -1)
    return torch.cat([y, x[..., rotary:]], -1)


def _levels(x):
    """Codes and fp16 scales of rows x [..., 128] in the rotated basis, one scale for each 64 channels."""
    x = x.unflatten(-1, (2, 64))
    scale = (x.abs().amax(-1).clamp(max=65504 * 7.5) / 7.5).to(torch.float16)
    d = scale.to(x.dtype)[..., None]
    code = torch.where(d > 0, (x / d + 8).floor().clamp(0, 15), 8.0)
    return code.flatten(-2).to(torch.uint8), scale


def _plain_append(s):
    c = s["case"]
    b, at = _rows(s)
    if s["q"] is not None:
        s["q_out"].copy_(_rope(s["q"], s, at, torch.float32))
    page, row = s["table"].long()[b, at // PAGE], at % PAGE
    k, v = _rope(s["k"], s, at, torch.float32).to(torch.bfloat16), s["v"]
    if c["op"] == "append_bf16":
        s["k_pages"][page, :, row] = k
        s["v_pages"][page, :, row] = v
        return dict(q=s["q_out"], k=s["k_pages"], v=s["v_pages"])
    kc, ks = _levels(_hadamard(k.float()))
    vc, vs = _levels(_hadamard(v.float()))
    ka, k_shift, va, v_shift, ksa, vsa = _places(s, row)
    flat = s["pages"].view(-1)
    base = (page[:, None] * c["hkv"] + torch.arange(c["hkv"], device=page.device)) * BLOCK
    for code, place, shift in ((kc, ka, k_shift), (vc, va, v_shift)):
        low, high = torch.nonzero(shift == 0).view(-1), torch.nonzero(shift).view(-1)
        low, high = low[place[0, low].argsort()], high[place[0, high].argsort()]  # the two nibbles of one byte
        flat[base[..., None] + place[:, None, low]] = code[..., low] | (code[..., high] << 4)
    for scale, place in ((ks, ksa), (vs, vsa)):
        s["pages"].view(torch.float16).view(-1)[(base[..., None] + place[:, None, :]) // 2] = scale
    return _plain_read(s, b, at)


def _held(s, page, row, dtype):
    """The rows that the 4-bit cache holds at (page, row) [m]: K and V [m, heads, 128] in the rotated basis."""
    hkv = s["case"]["hkv"]
    ka, k_shift, va, v_shift, ksa, vsa = _places(s, row)
    base = (page[:, None] * hkv + torch.arange(hkv, device=page.device)) * BLOCK
    flat, halves = s["pages"].view(-1), s["pages"].view(torch.float16).view(-1)

    def values(place, shift, scales):
        code = (flat[base[..., None] + place[:, None, :]] >> shift.to(torch.uint8)) & 15
        scale = halves[(base[..., None] + scales[:, None, :]) // 2].to(dtype)
        return ((code.to(dtype) - 7.5).unflatten(-1, (2, 64)) * scale[..., None]).flatten(-2)

    return values(ka, k_shift, ksa), values(va, v_shift, vsa)


def _plain_read(s, b, at):
    page, row = s["table"].long()[b, at // PAGE], at % PAGE
    k, v = _held(s, page, row, torch.float32)
    s["k_pages"][page, :, row] = _hadamard(k).to(torch.bfloat16)
    s["v_pages"][page, :, row] = _hadamard(v).to(torch.bfloat16)
    return dict(q=s.get("q_out"), k=s["k_pages"], v=s["v_pages"])


def _plain_attend(s):
    """Queries in blocks of consecutive tokens of a request; each block gathers the keys that any of its queries sees."""
    c = s["case"]
    dev = s["pos"].device
    hq, hkv, batch = c["hq"], c["hkv"], c["batch"]
    rows = 64 if s["most"] > 1 else 1
    blocks = -(-s["most"] // rows)
    window = c["window"] if c["window"] >= 0 else s["longest"]
    sinks = min(c["sinks"], s["longest"])
    i = torch.arange(blocks * rows, device=dev)
    first, length = s["pos"].long(), s["length"].long()
    p = (first[:, None] + i).view(batch, blocks, rows)                      # positions of the queries
    real = (i[None, :] < s["count"].long()[:, None]).view(batch, blocks, rows)
    token = (s["cu"].long()[:batch, None] + i).view(batch, blocks, rows)
    low = (p[:, :, 0] - window + 1).clamp(min=sinks)
    span = min(window + rows - 1, s["longest"])
    at = torch.cat([torch.arange(sinks, device=dev).expand(batch, blocks, sinks),
                    low[..., None] + torch.arange(span, device=dev)], -1)   # positions of the gathered keys
    held = at < length[:, None, None]
    page = s["table"].long().clamp(min=0)[torch.arange(batch, device=dev)[:, None, None],
                                          (at // PAGE).clamp(max=s["table"].shape[1] - 1)]
    if c["op"] == "attend_int4":
        k, v = [t.view(batch * blocks, -1, hkv, D).transpose(1, 2)
                for t in _held(s, page.reshape(-1), (at % PAGE).reshape(-1), torch.float32)]
    else:
        k, v = [t[page, :, at % PAGE].float().view(batch * blocks, -1, hkv, D).transpose(1, 2)
                for t in (s["k_pages"], s["v_pages"])]
    sees = (held[:, :, None, :] & (at[:, :, None, :] <= p[..., None])
            & ((at[:, :, None, :] < sinks) | (at[:, :, None, :] > p[..., None] - window)))
    sees = sees & real[..., None]
    q = s["q"].float()[token.clamp(max=max(s["n"] - 1, 0)).view(-1)]
    if c["op"] == "attend_int4":
        q = _hadamard(q)
    group = hq // hkv
    q = q.view(batch * blocks, rows, hkv, group, D).permute(0, 2, 3, 1, 4).reshape(batch * blocks, hkv, group * rows, D)
    x = (q @ k.transpose(-1, -2)) * (1.0 / math.sqrt(D))
    mask = sees.view(batch * blocks, 1, 1, rows, -1).expand(-1, hkv, group, -1, -1).reshape(x.shape)
    x = x.masked_fill(~mask, -torch.inf)
    top = x.amax(-1, keepdim=True)
    e = torch.exp(x - torch.where(top == -torch.inf, 0.0, top))
    y = (e @ v) / e.sum(-1, keepdim=True).clamp(min=1e-30)
    if c["op"] == "attend_int4":
        y = _hadamard(y)
    y = y.view(batch * blocks, hkv, group, rows, D).permute(0, 3, 1, 2, 4).reshape(-1, hq, D)
    keep = real.view(-1)
    s["out"][token.view(-1)[keep]] = y[keep].to(torch.bfloat16)
    return dict(out=s["out"])


def run(state):
    if own:
        return _own(state)
    op = state["case"]["op"]
    if op.startswith("append"):
        return _plain_append(state)
    if op == "read_int4":
        i = torch.arange(state["longest"], device=state["pos"].device)
        b, at = torch.nonzero(i[None, :] < state["length"].long()[:, None], as_tuple=True)
        return _plain_read(state, b, at)
    return _plain_attend(state)


# ---------------------------------------------------------------- bytes and operations


def work(case):
    first, count, length = _spans(case)
    hq, hkv = case["hq"], case["hkv"]
    n, op = int(count.sum()), case["op"]
    row = D * 2                       # one BF16 row of a head
    held = TILE_BYTES / TILE          # one token's K and V of a head in 4 bits
    if op.startswith("append"):
        table = case["rotary"] * 4
        values = n * (2 * hq + 2 * hkv) * row + n * table
        values += n * hkv * (2 * row if op == "append_bf16" else held)
        flops = n * (hq + hkv) * case["rotary"] * 3
        if op == "append_int4":       # the 128-point transforms, there and back
            values += n * hkv * (held + 2 * row)
            flops += n * hkv * 2 * 2 * 7 * D
        return {"bytes": float(values), "flops": float(flops)}
    if op == "read_int4":
        t = int(length.sum())
        return {"bytes": float(t * hkv * (held + 2 * row)), "flops": float(t * hkv * 2 * 7 * D)}
    pairs = keys = 0
    for f, c, e in zip(first.tolist(), count.tolist(), length.tolist()):
        p = np.arange(f, f + c)
        low = np.maximum(p - case["window"] + 1, 0) if case["window"] >= 0 else np.zeros_like(p)
        pairs += int((np.minimum(p + 1, e) - low + np.minimum(case["sinks"], low)).sum())
        keys += e - int(low[0]) + min(case["sinks"], int(low[0]))
    token = held if op == "attend_int4" else 2 * row
    return {"bytes": float(keys * hkv * token + 2 * n * hq * row), "flops": float(4 * pairs * hq * D)}


# ---------------------------------------------------------------- the definitions in 64 bits


def _transform():
    """The 128-point Hadamard matrix by doubling, over sqrt(128)."""
    m = np.ones((1, 1))
    while m.shape[0] < D:
        m = np.block([[m, m], [m, -m]])
    return torch.from_numpy(m / math.sqrt(D)).cuda()


def _turned(x, s, at):
    """Each rotated pair as a complex number times cos + i sin."""
    rotary, x = s["case"]["rotary"], x.double()
    if not rotary:
        return x
    table = s["rope"].double()[at]
    turn = torch.complex(table[:, : rotary // 2], table[:, rotary // 2:])[:, None, :]
    head = x[..., :rotary]
    if s["case"]["interleaved"]:
        z = torch.view_as_complex(head.unflatten(-1, (rotary // 2, 2)).contiguous()) * turn
        head = torch.view_as_real(z).flatten(-2)
    else:
        z = torch.complex(head[..., : rotary // 2].contiguous(), head[..., rotary // 2:].contiguous()) * turn
        head = torch.cat([z.real, z.imag], -1)
    return torch.cat([head, x[..., rotary:]], -1)


def _through_4_bits(x):
    """What rows x [..., 128] (64 bits, original basis) become in the cache."""
    m = _transform()
    y = (x @ m).unflatten(-1, (2, 64))
    scale = (y.abs().amax(-1, keepdim=True).clamp(max=65504 * 7.5) / 7.5).to(torch.float16).double()
    code = torch.floor(y / torch.where(scale > 0, scale, 1.0) + 8).clamp(0, 15)
    return ((code - 7.5) * scale).flatten(-2) @ m


def _unpacked(s, block_of, n):
    """K and V [heads, n, 128] of positions 0..n-1 held in the blocks block_of [pages, heads, BLOCK], original basis."""
    tiles = block_of.unflatten(-1, (4, TILE_BYTES)).transpose(0, 1).flatten(1, 2)[:, : -(-n // TILE)]
    heads = tiles.shape[0]
    scale = tiles[..., 2048:].contiguous().view(torch.float16).view(heads, -1, 2, TILE, 2).double()
    code = torch.stack([tiles[..., :2048] & 15, tiles[..., :2048] >> 4], -1).view(heads, tiles.shape[1], 2, 2048)
    # K: nibbles [token][channel bits 4,3][bits 6,5][bit 0][bit 2][bit 1]
    k = code[:, :, 0].view(heads, -1, TILE, 4, 4, 2, 2, 2).permute(0, 1, 2, 4, 3, 6, 7, 5).reshape(heads, -1, TILE, D)
    # V: [bit 6][bit 3][bits 1,0][token bits 2,1][bit 5][bit 2][token bit 0][token bit 3][bit 4]
    v = code[:, :, 1].view(heads, -1, 2, 2, 4, 4, 2, 2, 2, 2, 2)
    v = v.permute(0, 1, 9, 5, 8, 2, 6, 10, 3, 7, 4).reshape(heads, -1, TILE, D)
    m = _transform()

    def values(c, sc):
        return (((c.double() - 7.5).unflatten(-1, (2, 64)) * sc[..., None]).flatten(-2) @ m).flatten(1, 2)[:, :n]

    return values(k, scale[:, :, 0]), values(v, scale[:, :, 1])


def exact(case, seed):
    s = prepare(case, seed)
    op, hkv, hq = case["op"], case["hkv"], case["hq"]
    first, count, length = _spans(case)
    table = s["table"].long()
    if op.startswith("append"):
        at = torch.from_numpy(np.concatenate([np.arange(f, f + c) for f, c in zip(first, count)])).cuda()
        b = torch.from_numpy(np.repeat(np.arange(case["batch"]), count)).cuda()
        k = _turned(s["k"], s, at).to(torch.bfloat16).double()
        v = s["v"].double()
        if op == "append_int4":
            k, v = _through_4_bits(k), _through_4_bits(v)
        out = {}
        if s["q"] is not None:
            out["q"] = _turned(s["q"], s, at)
        for name, x in (("k", k), ("v", v)):
            pages = s[name + "_pages"].double()
            pages[table[b, at // PAGE], :, at % PAGE] = x
            out[name] = pages
        return out
    if op == "read_int4":
        out = {name: s[name + "_pages"].double() for name in "kv"}
        for r in range(case["batch"]):
            n = int(length[r])
            ids = table[r, : -(-n // PAGE)]
            at = torch.arange(n, device="cuda")
            for name, x in zip("kv", _unpacked(s, s["pages"][ids], n)):
                out[name][ids[at // PAGE], :, at % PAGE] = x.transpose(0, 1)
        return out
    if 4.0 * D * hq * float(sum(int(c) * (int(e) if case["window"] < 0 else min(int(e), case["window"] + case["sinks"] + int(c)))
                                for c, e in zip(count, length))) > 8e12:
        return None
    out = torch.zeros((s["n"], hq, D), dtype=torch.float64, device="cuda")
    begin = 0
    for r in range(case["batch"]):
        n, f, c = int(length[r]), int(first[r]), int(count[r])
        ids = table[r, : -(-n // PAGE)].clamp(min=0)
        if op == "attend_int4":
            k, v = _unpacked(s, s["pages"][ids], n)
        else:
            k, v = [s[name][ids].double().transpose(0, 1).flatten(1, 2)[:, :n] for name in ("k_pages", "v_pages")]
        for lo in range(0, c, 2048):
            p = torch.arange(f + lo, f + min(c, lo + 2048), device="cuda")
            at = torch.arange(n, device="cuda")
            if case["window"] >= 0:  # keys that none of these queries sees are left out
                at = at[(at < case["sinks"]) | (at > f + lo - case["window"])]
            at = at[at <= int(f + min(c, lo + 2048) - 1)]
            sees = at[None, :] <= p[:, None]
            if case["window"] >= 0:
                sees &= (at[None, :] < case["sinks"]) | (p[:, None] - at[None, :] < case["window"])
            for h in range(hkv):
                q = s["q"][begin + lo: begin + lo + len(p), h * (hq // hkv): (h + 1) * (hq // hkv)].double()
                x = torch.einsum("nhd,td->hnt", q, k[h, at]) / math.sqrt(D)
                w = torch.softmax(torch.where(sees, x, -torch.inf), -1)
                out[begin + lo: begin + lo + len(p), h * (hq // hkv): (h + 1) * (hq // hkv)] = torch.einsum(
                    "hnt,td->nhd", w, v[h, at])
        begin += c
    return {"out": out}
