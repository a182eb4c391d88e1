"""Cases and plain forms of the operators of a prompt on its way into the mixed INT2 cache: the table of positions
scaled for long contexts, the rotation of queries and keys by it, the attention over whole prompts in packed rows,
and the read-back of the mixed cache into BF16 pages.

``listed()`` and ``draw()`` name cases, ``prepare()`` makes a case's inputs on the GPU, ``run()`` makes one pass:
with ``own`` the framework's calls, otherwise the same operators in elementary torch operations.  ``exact()`` is
the operator's definition in 64 bits.
"""

import math

import numpy as np
import torch

own = False

D = 128       # channels of a head
PAGE = 64     # tokens of a page
SINK = 64     # first tokens that stay BF16 in the mixed cache
RECENT = 256  # last tokens that do
BLOCK = 4608  # one page of one head in 2 bits: K codes 2048 | K scales 256 | V codes 2048 | V scales 256

# ---------------------------------------------------------------- cases


def listed():
    return [
        # a model's table for 131,072 positions, stretched from 32,768 by the ramp over channels; made when it is loaded
        dict(name="table_index_131k", op="table", positions=131072, rotary=128, theta=1.0e6, scaling="index", factor=4.0,
             original=32768),
        # a small model's, by the ramp over turns
        dict(name="table_turns_8k", op="table", positions=8192, rotary=64, theta=5.0e5, scaling="turns", factor=8.0,
             original=2048),
        # one decode step's queries and keys of 64 requests, from a fused projection, ahead of the step over the INT2 cache
        dict(name="rotate_step", op="rotate", hq=32, hkv=8, batch=64, tokens=1, first=131000, rotary=128, interleaved=False,
             inverse=False, dtype="bf16", fused=True),
        # four prompts of uneven length prefilled together; three quarters of the channels, as adjacent pairs
        dict(name="rotate_prompts", op="rotate", hq=64, hkv=8, batch=4, tokens=8192, first=0, rotary=96, interleaved=True,
             inverse=False, dtype="bf16", fused=True),
        # a calibration set's captured queries and keys in 32 bits, turned back to where they were before their positions
        dict(name="rotate_calibration", op="rotate", hq=32, hkv=8, batch=1, tokens=16384, first=0, rotary=128,
             interleaved=False, inverse=True, dtype="fp32", fused=False),
        # the smallest call: one short prompt of a small model
        dict(name="attend_short", op="attend", hq=8, hkv=2, batch=1, tokens=37, kept=0, window=-1, sinks=0, fused=True),
        # a prefill batch of prompts of 1 to 2048 tokens
        dict(name="attend_batch", op="attend", hq=32, hkv=8, batch=48, tokens=2048, kept=0, window=-1, sinks=0, fused=True),
        # one long prompt
        dict(name="attend_long", op="attend", hq=32, hkv=8, batch=1, tokens=24001, kept=0, window=-1, sinks=0, fused=False),
        # prompts through a windowed layer, eight query heads to a KV head
        dict(name="attend_window", op="attend", hq=64, hkv=8, batch=3, tokens=12288, kept=0, window=4096, sinks=64,
             fused=True),
        # the next 300 tokens or less of two conversations whose earlier rows were kept
        dict(name="attend_more", op="attend", hq=32, hkv=8, batch=2, tokens=300, kept=40000, window=-1, sinks=0, fused=False),
        # a serving batch's prefixes, short and ragged, some without any quantised token yet
        dict(name="read_batch", op="read", hkv=8, batch=28, lo=100, hi=4096, part=True),
        # a chunk's whole prefix out of the INT2 cache
        dict(name="read_100k", op="read", hkv=8, batch=1, lo=99991, hi=99991, part=False),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["table", "rotate", "rotate", "attend", "attend", "attend", "read", "read"])
    if op == "table":
        return dict(op=op, positions=_log(rng, 1, 131072), rotary=16 * rng.randint(1, 8), theta=float(_log(rng, 1e4, 1e7)),
                    scaling=rng.choice(["none", "linear", "ntk", "turns", "index", "factors"]),
                    factor=round(rng.uniform(1.5, 32.0), 2), original=_log(rng, 2048, 65536))
    hkv = rng.choice([1, 2, 4, 8])
    hq = hkv * rng.choice([1, 2, 4, 5, 8])
    step = rng.random() < 0.4
    if op == "rotate":
        batch = _log(rng, 1, 64) if step else _log(rng, 1, 6)
        fp32 = rng.random() < 0.3
        tokens = 1 if step else _log(rng, 2, (16384 if fp32 else 32768) // batch)
        return dict(op=op, hq=hq, hkv=hkv, batch=batch, tokens=tokens, first=_log(rng, 1, 100000), rotary=16 * rng.randint(1, 8),
                    interleaved=rng.random() < 0.5, inverse=rng.random() < 0.3, dtype="fp32" if fp32 else "bf16",
                    fused=rng.random() < 0.5)
    if op == "read":
        batch = _log(rng, 1, 32)
        hi = _log(rng, 1, 100000 // batch)
        return dict(op=op, hkv=hkv, batch=batch, lo=max(1, hi // 8), hi=hi, part=rng.random() < 0.5)
    window = -1 if rng.random() < 0.6 else _log(rng, 1, 8192)
    sinks = rng.choice([0, 1, 4, 64, rng.randint(1, 200)]) if window >= 0 else 0
    more = rng.random() < 0.4
    batch = _log(rng, 1, 48)
    tokens = (1 if step else _log(rng, 2, 2048 // batch)) if more else _log(rng, 1, 16384 // batch)
    return dict(op=op, hq=hq, hkv=hkv, batch=batch, tokens=tokens, kept=_log(rng, 1, 65536 // batch) if more else 0,
                window=window, sinks=sinks, fused=rng.random() < 0.5 and not more)


def _spans(case):
    """Each request's new tokens and the positions that come before them, on the host: the case's own, whatever the seed."""
    n = case["batch"]
    r = np.random.RandomState(n + case.get("tokens", 0))
    if case["op"] == "read":
        length = r.randint(case["lo"], case["hi"] + 1, n).astype(np.int64)
        length[r.randint(n)] = case["hi"]
        first = (length * r.random_sample(n) * 0.3).astype(np.int64) if case["part"] else np.zeros_like(length)
        return first, length - first, length  # from, how many, held
    t = case["tokens"]
    count = np.full(n, t, np.int64)
    if n > 1 and t > 1:
        lo = 1 if case["op"] == "attend" else max(1, t // 2)
        count = r.randint(lo, t + 1, n).astype(np.int64)
        count[r.randint(n)] = t
    before = case["kept"] if case["op"] == "attend" else case["first"]
    first = r.randint(before // 2, before + 1, n).astype(np.int64)
    return first, count, first + count


def _frequencies(case):
    """The scaled frequencies (64 bits, host) and the amplitude of a table."""
    d, s, theta = case["rotary"], case["factor"], case["theta"]
    i = np.arange(d // 2, dtype=np.float64)
    f = theta ** (-2.0 * i / d)
    kind = case["scaling"]
    if kind == "linear":
        return f / s, 1.0
    if kind == "ntk":
        return f * s ** (-2.0 * i / (d - 2)), 1.0
    if kind == "turns":
        turns = case["original"] * f / (2 * math.pi)
        g = np.clip((turns - 1.0) / (4.0 - 1.0), 0, 1)
        return f * ((1 - g) / s + g), 1.0
    if kind == "index":
        place = lambda turns: d * math.log(case["original"] / (2 * math.pi * turns)) / (2 * math.log(theta))  # noqa: E731
        lo, hi = max(0, math.floor(place(32.0))), min(d - 1, math.ceil(place(1.0)))
        g = 1 - np.clip((i - lo) / max(hi - lo, 1e-3), 0, 1)
        return f * ((1 - g) / s + g), 0.1 * math.log(s) + 1
    if kind == "factors":
        return f / _factors(case), 1.0
    return f, 1.0


def _factors(case):
    """A divisor for each frequency, growing towards the slow ones."""
    half = case["rotary"] // 2
    return 1.0 + (case["factor"] - 1.0) * (np.arange(half) + 1.0) / half


def _rotation():
    """A fixed orthogonal U and the layer's rotation R = U H P (64 bits, host)."""
    u = np.linalg.qr(np.random.RandomState(7).standard_normal((D, D)))[0].astype(np.float32)
    i = np.arange(D)
    h = 1.0 - 2.0 * (np.array([bin(x).count("1") for x in (i[:, None] & i[None, :]).ravel()]).reshape(D, D) & 1)
    reverse = np.array([int(format(x, "07b")[::-1], 2) for x in i])
    return u, (u.astype(np.float64) @ h / math.sqrt(D))[:, reverse]


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    dev = torch.device("cuda")
    if case["op"] == "table":
        # (the seed moves the base a little: a table has no other input)
        theta = case["theta"] * (1.0 + 0.001 * np.random.RandomState(seed % (1 << 31)).random_sample())
        return dict(case=dict(case, theta=theta),
                    table=torch.zeros((case["positions"], case["rotary"]), dtype=torch.float32, device=dev))
    first, count, end = _spans(case)
    batch, hkv = case["batch"], case["hkv"]
    ints = lambda x: torch.from_numpy(np.ascontiguousarray(x, dtype=np.int32)).to(dev)  # noqa: E731
    starts = lambda x: np.concatenate([[0], np.cumsum(x)])  # noqa: E731
    s = dict(case=case, first=first, counts=count, end=end, n=int(count.sum()), most=int(count.max()), longest=int(end.max()),
             pos=ints(first), count=ints(count), length=ints(end), cu=ints(starts(count)))

    def randn(*shape):
        return torch.randn(shape, generator=g, device=dev)

    def outliers(x):
        """Four channels of each head stand out by a factor of 20."""
        r = np.random.RandomState((seed + 2) % (1 << 31))
        scale = torch.ones(x.shape[-2:])
        for h in range(x.shape[-2]):
            scale[h, torch.from_numpy(r.choice(D, 4, replace=False))] = 20.0
        return x.mul_(scale.to(dev))

    if case["op"] == "read":
        logical = int(-(-s["longest"] // PAGE))
        held = np.arange(logical)[None, :] * PAGE < end[:, None]
        n_pages = int(held.sum()) + 1
        r = np.random.RandomState((seed + 1) % (1 << 31))
        tables = []
        for _ in range(2):  # the INT2 pages' and the BF16 pages'
            t = np.full(held.shape, -1, np.int32)
            t[held] = r.permutation(n_pages)[: n_pages - 1]
            tables.append(ints(t))
        shape = (n_pages, hkv, BLOCK)
        a, b = [torch.randint(0, 256, shape, dtype=torch.uint8, device=dev, generator=g) for _ in range(2)]
        low = (((a & 0x33) + (b & 0x33)) >> 1) & 0x33
        high = ((((a >> 2) & 0x33) + ((b >> 2) & 0x33) + 0x11) >> 1) & 0x33
        pages = low | (high << 2)
        for at in (2048, 4352):
            scale = randn(n_pages, hkv, PAGE * 2).mul_(0.25).exp_().mul_(0.8).to(torch.float16)
            pages[..., at: at + 256] = scale.view(torch.uint8)
        s.update(int2=pages, from_table=tables[0], to_table=tables[1], sink_page=ints(r.permutation(batch)),
                 ring_slot=ints(r.permutation(batch)))
        for name in "kv":
            s[name + "_sink"] = outliers(randn(batch, PAGE, hkv, D)).to(torch.bfloat16).transpose(1, 2).contiguous()
            s[name + "_ring"] = outliers(randn(batch, RECENT, hkv, D)).to(torch.bfloat16).transpose(1, 2).contiguous()
            s[name + "_pages"] = torch.zeros((n_pages, hkv, PAGE, D), dtype=torch.bfloat16, device=dev)
        s["u"], rotation = _rotation()
        s["rotation"] = torch.from_numpy(rotation).to(dev)
        return s

    hq, n = case["hq"], s["n"]
    keys = n + int(first.sum()) if case["op"] == "attend" else n
    dtype = torch.float32 if case.get("dtype") == "fp32" else torch.bfloat16
    heads = [hq, hkv, hkv]
    rows = [n, keys, keys]
    x = [randn(r, h, D) for r, h in zip(rows, heads)]
    x[1:] = [outliers(t) for t in x[1:]]
    x = [t.to(dtype).view(r, -1) for t, r in zip(x, rows)]
    if case["fused"]:  # views of one projection's output
        x = list(torch.cat(x, 1).split([h * D for h in heads], 1))
    s["q"], s["k"], s["v"] = [t.unflatten(1, (h, D)) for t, h in zip(x, heads)]
    if case["op"] == "rotate":
        s["q_out"], s["k_out"] = [torch.zeros((n, h, D), dtype=dtype, device=dev) for h in (hq, hkv)]
        del s["v"]
        half = case["rotary"] // 2
        angle = torch.arange(s["longest"], dtype=torch.float64, device=dev)[:, None] * (
            1.0e6 ** (-torch.arange(half, dtype=torch.float64, device=dev) / half))[None, :]
        s["rope"] = torch.cat([angle.cos(), angle.sin()], 1).to(torch.float32)
    else:
        s["cu_k"] = ints(starts(end))
        s["out"] = torch.zeros((n, hq, D), dtype=torch.bfloat16, device=dev)
    return s


# ---------------------------------------------------------------- the framework's calls

_contexts = {}  # one library handle for each head shape, as a user's program keeps it


def _plan(s):
    """The views, argument blocks and workspace that a user's program makes once for its tensors."""
    from int2_rotated_kv_oscar_gb300 import abi
    from int2_rotated_kv_oscar_gb300 import cache as kv
    c = s["case"]
    heads = (c.get("hq") or c.get("hkv", 1), c.get("hkv", 1))
    if heads not in _contexts:
        _contexts[heads] = abi.oscar_create(abi.oscar_config(
            num_layers=1, num_q_heads=heads[0], num_kv_heads=heads[1], head_dim=D, page_size=PAGE, sink=SINK,
            recent=RECENT, group=64, device=torch.cuda.current_device()))
    p = dict(ctx=_contexts[heads], abi=abi)
    if c["op"] == "table":
        p["scaling"] = None if c["scaling"] == "none" else kv.rope_scaling(
            c["scaling"], c["factor"], original_positions=c["original"],
            factors=_factors(c) if c["scaling"] == "factors" else None)
    elif c["op"] == "rotate":
        p["args"] = kv.rope_args(s["rope"], s["pos"], q=s["q"], q_out=s["q_out"], k=s["k"], k_out=s["k_out"],
                                 interleaved=c["interleaved"], inverse=c["inverse"],
                                 cu_seqlens=s["cu"] if s["most"] > 1 else None, max_tokens_per_req=s["most"])
    elif c["op"] == "attend":
        p["args"] = kv.prompt_args(s["q"], s["k"], s["v"], s["out"], s["cu"], s["most"],
                                   cu_seqlens_k=s["cu_k"] if c["kept"] else None,
                                   max_keys_per_req=s["longest"] if c["kept"] else None, window=c["window"],
                                   sinks=c["sinks"])
        p["workspace"] = kv.window_workspace(p["ctx"])
    else:
        abi.oscar_load_rotation(p["ctx"], 0, s["u"], s["u"], 30.0, 30.0)
        p["from"] = abi.oscar_cache_view(
            int2_pages=s["int2"].data_ptr(), num_pages=s["int2"].shape[0], k_sink=s["k_sink"].data_ptr(),
            v_sink=s["v_sink"].data_ptr(), num_sink_pages=c["batch"], k_ring=s["k_ring"].data_ptr(),
            v_ring=s["v_ring"].data_ptr(), num_ring_slots=c["batch"], page_table=s["from_table"].data_ptr(),
            max_pages_per_req=s["from_table"].shape[1], sink_page=s["sink_page"].data_ptr(),
            ring_slot=s["ring_slot"].data_ptr(), batch=c["batch"], recent_page_table=None)
        p["to"] = kv.bf16_view(s["k_pages"], s["v_pages"], s["to_table"])
    return p


def _own(s):
    p = s.get("plan")
    if p is None:
        p = s["plan"] = _plan(s)
    abi, ctx, c = p["abi"], p["ctx"], s["case"]
    stream = torch.cuda.current_stream()
    if c["op"] == "table":
        abi.oscar_rope_table_scaled(ctx, s["table"], c["theta"], p["scaling"], stream)
        return dict(table=s["table"])
    if c["op"] == "rotate":
        abi.oscar_rope_rotate(ctx, p["args"], stream)
        return dict(q=s["q_out"], k=s["k_out"])
    if c["op"] == "attend":
        _, pointer, size = p["workspace"]
        abi.oscar_prompt_attention(ctx, p["args"], pointer, size, stream)
        return dict(out=s["out"])
    abi.oscar_int2_to_bf16(ctx, 0, p["from"], p["to"], s["length"], s["pos"], s["count"], s["most"], stream)
    return dict(k=s["k_pages"], v=s["v_pages"])


# ---------------------------------------------------------------- the plain forms


def _plain_table(s):
    """Angles, cosines and sines in 64 bits (a far position's angle needs more than 24), rounded once."""
    f, amplitude = _frequencies(s["case"])
    n, half = s["case"]["positions"], s["case"]["rotary"] // 2
    p = torch.arange(n, dtype=torch.float64, device=s["table"].device)
    angle = p[:, None] * torch.from_numpy(f).to(p.device)[None, :]
    s["table"][:, :half] = (torch.cos(angle) * amplitude).to(torch.float32)
    s["table"][:, half:] = (torch.sin(angle) * amplitude).to(torch.float32)
    return dict(table=s["table"])


def _rows(s):
    """The position of every new token."""
    i = torch.arange(s["n"], device=s["cu"].device)
    b = (torch.searchsorted(s["cu"].long(), i, right=True) - 1).clamp(0, s["case"]["batch"] - 1)
    return s["pos"].long()[b] + i - s["cu"].long()[b]


def _plain_rotate(s):
    c = s["case"]
    half = c["rotary"] // 2
    row = s["rope"][_rows(s)][:, None, :]
    cos, sin = row[..., :half], row[..., half:]
    if c["inverse"]:
        sin = -sin
    for name in "qk":
        x, y = s[name].float(), s[name + "_out"]
        pairs = (slice(0, c["rotary"], 2), slice(1, c["rotary"], 2)) if c["interleaved"] else (
            slice(0, half), slice(half, c["rotary"]))
        a, b = x[..., pairs[0]], x[..., pairs[1]]
        y[..., pairs[0]] = (a * cos - b * sin).to(y.dtype)
        y[..., pairs[1]] = (b * cos + a * sin).to(y.dtype)
        y[..., c["rotary"]:] = s[name][..., c["rotary"]:]
    return dict(q=s["q_out"], k=s["k_out"])


def _plain_attend(s):
    """One request after the other, its queries in blocks, each over the keys that any of them sees."""
    c = s["case"]
    dev, group = s["q"].device, c["hq"] // c["hkv"]
    row = key = 0
    for first, count, end in zip(s["first"].tolist(), s["counts"].tolist(), s["end"].tolist()):
        step = max(16, min(1024, (1 << 29) // (end * c["hq"])))
        for lo in range(0, count, step):
            n = min(step, count - lo)
            p = torch.arange(first + lo, first + lo + n, device=dev)
            last, begin = first + lo + n, 0
            if c["window"] >= 0:
                begin = max(min(c["sinks"], last), first + lo - c["window"] + 1)
            at = torch.arange(begin, last, device=dev)
            if c["window"] >= 0 and begin > 0:
                at = torch.cat([torch.arange(min(c["sinks"], begin), device=dev), at])
            sees = at[None, :] <= p[:, None]
            if c["window"] >= 0:
                sees &= (at[None, :] < c["sinks"]) | (at[None, :] > p[:, None] - c["window"])
            k, v = [s[x][key + at].float().permute(1, 2, 0) for x in "kv"]
            q = s["q"][row + lo: row + lo + n].float().view(n, c["hkv"], group, D).permute(1, 2, 0, 3)
            x = (q.reshape(c["hkv"], group * n, D) @ k) * (1.0 / math.sqrt(D))
            x = x.view(c["hkv"], group, n, -1).masked_fill(~sees, -torch.inf)
            top = x.amax(-1, keepdim=True)
            x = torch.exp(x - torch.where(top == -torch.inf, 0.0, top))
            y = (x.view(c["hkv"], group * n, -1) @ v.transpose(1, 2)).view(c["hkv"], group, n, D)
            y = y / x.sum(-1, keepdim=True).clamp(min=1e-30)
            s["out"][row + lo: row + lo + n] = y.permute(2, 0, 1, 3).reshape(n, c["hq"], D).to(torch.bfloat16)
        row += count
        key += end
    return dict(out=s["out"])


def _places(t):
    """Byte offsets in a block of the codes of tokens t (0..63), K and V [len(t), 128], and the shifts in the byte [128]."""
    j = torch.arange(D, device=t.device)
    tile, u = (512 * (t >> 4))[:, None], (t & 15)[:, None]
    k = tile + 64 * (u & 7) + 16 * ((j >> 2) & 3) + 8 * (u >> 3) + 4 * (j >> 6) + (j & 3)
    v = 2304 + tile + 64 * (j & 7) + 16 * ((u & 7) >> 1) + 8 * (u >> 3) + 4 * ((j >> 3) & 1) + 2 * (u & 1) + (j >> 6)
    return (k, 4 * ((j >> 5) & 1) + 2 * ((j >> 4) & 1)), (v, 2 * ((j >> 4) & 3))


def _plain_read(s):
    c = s["case"]
    dev, heads = s["pos"].device, c["hkv"]
    i = torch.arange(s["longest"], device=dev)
    wanted = (i >= s["pos"][:, None]) & (i < (s["pos"] + s["count"])[:, None])
    b, at = torch.nonzero(wanted, as_tuple=True)
    end = s["length"].long()[b]
    sink, recent = at < SINK, (at >= SINK) & (at >= end - RECENT)
    to = s["to_table"].long()[b, at // PAGE]
    h = ~(sink | recent)
    base = (s["from_table"].long()[b[h], at[h] // PAGE][:, None] * heads + torch.arange(heads, device=dev)) * BLOCK
    turn = s["rotation"].float().T
    flat, halves = s["int2"].view(-1), s["int2"].view(torch.float16).view(-1)
    for name, (place, shift), scales in zip("kv", _places(at[h] % PAGE), (2048, 4352)):
        pages = s[name + "_pages"]
        pages[to[sink], :, at[sink] % PAGE] = s[name + "_sink"][s["sink_page"].long()[b[sink]], :, at[sink]]
        pages[to[recent], :, at[recent] % PAGE] = s[name + "_ring"][s["ring_slot"].long()[b[recent]], :, (at[recent] - SINK) % RECENT]
        if base.shape[0]:
            code = (flat[base[..., None] + place[:, None, :]] >> shift.to(torch.uint8)) & 3
            row = (base + scales + 4 * (at[h] % PAGE)[:, None])[..., None] // 2 + torch.arange(2, device=dev)
            x = ((code.float() - 1.5).unflatten(-1, (2, 64)) * halves[row].float()[..., None]).flatten(-2)
            pages[to[h], :, at[h] % PAGE] = (x @ turn).to(torch.bfloat16)
    return dict(k=s["k_pages"], v=s["v_pages"])


def run(state):
    if own:
        return _own(state)
    return dict(table=_plain_table, rotate=_plain_rotate, attend=_plain_attend, read=_plain_read)[state["case"]["op"]](state)


# ---------------------------------------------------------------- bytes and operations


def work(case):
    if case["op"] == "table":
        entries = case["positions"] * case["rotary"]
        return {"bytes": 4.0 * entries, "flops": 1.5 * entries}  # an angle, its cosine and sine for two entries
    first, count, end = _spans(case)
    n, hkv = int(count.sum()), case["hkv"]
    if case["op"] == "read":
        history = np.maximum(np.minimum(first + count, end - RECENT) - np.maximum(first, SINK), 0).sum()
        values = hkv * (n * 512 + history * 72 + (n - history) * 512)
        return {"bytes": float(values), "flops": float(history * hkv * 2 * 2 * D * D)}
    hq = case["hq"]
    if case["op"] == "rotate":
        size = 4 if case["dtype"] == "fp32" else 2
        return {"bytes": float(n * (2 * (hq + hkv) * D * size + 4 * case["rotary"])),
                "flops": float(n * (hq + hkv) * case["rotary"] * 3)}
    pairs = keys = 0
    for f, c, e in zip(first.tolist(), count.tolist(), end.tolist()):
        p = np.arange(f, f + c)
        low = np.maximum(p - case["window"] + 1, 0) if case["window"] >= 0 else np.zeros_like(p)
        pairs += int((p + 1 - low + np.minimum(case["sinks"], low)).sum())
        keys += e - int(low[0]) + min(case["sinks"], int(low[0]))
    return {"bytes": float(4 * (keys * hkv + n * hq) * D), "flops": float(4 * pairs * hq * D)}


# ---------------------------------------------------------------- the definitions in 64 bits


def _turned(x, s):
    """Each rotated pair as a complex number times cos + i sin, or its conjugate."""
    rotary = s["case"]["rotary"]
    at = torch.from_numpy(np.concatenate([np.arange(f, f + c) for f, c in zip(s["first"], s["counts"])])).to(x.device)
    table = s["rope"].double()[at]
    turn = torch.complex(table[:, : rotary // 2], table[:, rotary // 2:])[:, None, :]
    if s["case"]["inverse"]:
        turn = turn.conj()
    x = x.double()
    head = x[..., :rotary]
    if s["case"]["interleaved"]:
        head = torch.view_as_real(torch.view_as_complex(head.unflatten(-1, (rotary // 2, 2)).contiguous()) * turn).flatten(-2)
    else:
        z = torch.complex(head[..., : rotary // 2].contiguous(), head[..., rotary // 2:].contiguous()) * turn
        head = torch.cat([z.real, z.imag], -1)
    return torch.cat([head, x[..., rotary:]], -1)


def _held(s, r):
    """What request r's positions stand for, K and V [heads, length, 128]."""
    n, hkv = int(s["end"][r]), s["case"]["hkv"]
    ids = s["from_table"][r, : -(-n // PAGE)].long()
    blocks = s["int2"][ids].transpose(0, 1)  # [heads, pages, BLOCK]
    p = torch.arange(n, device=ids.device)
    out = []
    # the bits of token u and channel j in the order of a code area's bytes and 2-bit fields, and back to (u, j)
    for name, at, dims, order in (("k", 0, (4, 8, 4, 2, 2, 4, 2, 2), (0, 3, 1, 4, 6, 7, 2, 5)),
                                  ("v", 2304, (4, 8, 4, 2, 2, 2, 2, 2, 2), (0, 3, 2, 5, 6, 7, 8, 4, 1))):
        area = blocks[..., at: at + 2048]
        code = torch.stack([(area >> (2 * f)) & 3 for f in range(4)], -1)
        code = code.reshape(hkv, -1, *dims).permute(0, 1, *[2 + o for o in order]).reshape(hkv, -1, D).double()
        scale = blocks[..., at + 2048: at + 2304].contiguous().view(torch.float16).reshape(hkv, -1, 2).double()
        x = ((code - 1.5).unflatten(-1, (2, 64)) * scale[..., None]).flatten(-2)[:, :n] @ s["rotation"].transpose(0, 1)
        ring = s[name + "_ring"][int(s["ring_slot"][r])].double()
        late = p[max(SINK, n - RECENT):]
        x[:, late] = ring[:, (late - SINK) % RECENT]
        early = p[:SINK]
        x[:, early] = s[name + "_sink"][int(s["sink_page"][r])].double()[:, early]
        out.append(x)
    return out


def exact(case, seed):
    s = prepare(case, seed)
    case = s["case"]
    if case["op"] == "table":
        f, amplitude = _frequencies(case)
        angle = torch.outer(torch.arange(case["positions"], dtype=torch.float64), torch.from_numpy(f)).cuda()
        return {"table": amplitude * torch.view_as_real(torch.polar(torch.ones_like(angle), angle)).transpose(1, 2).flatten(1)}
    if case["op"] == "rotate":
        return {"q": _turned(s["q"], s), "k": _turned(s["k"], s)}
    if case["op"] == "read":
        out = {name: s[name + "_pages"].double() for name in "kv"}
        for r in range(case["batch"]):
            at = torch.arange(int(s["first"][r]), int(s["first"][r] + s["counts"][r]), device="cuda")
            page = s["to_table"][r].long()[at // PAGE]
            for name, x in zip("kv", _held(s, r)):
                out[name][page, :, at % PAGE] = x[:, at].transpose(0, 1)
        return out
    hq, hkv = case["hq"], case["hkv"]
    if work(case)["flops"] > 6e12:
        return None
    out = torch.zeros((s["n"], hq, D), dtype=torch.float64, device="cuda")
    row = key = 0
    for first, count, end in zip(s["first"].tolist(), s["counts"].tolist(), s["end"].tolist()):
        for lo in range(0, count, 2048):
            p = torch.arange(first + lo, first + min(count, lo + 2048), device="cuda")
            at = torch.arange(int(p[-1]) + 1, device="cuda")
            if case["window"] >= 0:  # keys that none of these queries sees are left out
                at = at[(at < case["sinks"]) | (at > first + lo - case["window"])]
            far = p[:, None] - at[None, :]
            sees = far >= 0
            if case["window"] >= 0:
                sees &= (at[None, :] < case["sinks"]) | (far < case["window"])
            mine = slice(row + lo, row + lo + len(p))
            for h in range(hkv):
                q = s["q"][mine, h * (hq // hkv): (h + 1) * (hq // hkv)].double()
                x = torch.einsum("nhd,td->hnt", q, s["k"][key + at, h].double()) / math.sqrt(D)
                x = torch.where(sees, x, -torch.inf)
                w = torch.where(sees.any(-1)[:, None], torch.softmax(x, -1), 0.0)
                out[mine, h * (hq // hkv): (h + 1) * (hq // hkv)] = torch.einsum("hnt,td->nhd", w, s["v"][key + at, h].double())
        row += count
        key += end
    return {"out": out}
