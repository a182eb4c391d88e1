"""Position rotation, the 4-bit cache and windowed attention, in fp64 (plain definitions, no layout tricks).

Rotation: pair (x, y) of a row at position p with frequency f_i = theta^(-2 i / rotary_dim) becomes
(x cos - y sin, y cos + x sin) of the angle p f_i; pairs are (i, i + rotary_dim / 2) or (2 i, 2 i + 1).
4-bit cache: x' = x H / sqrt(128) (Sylvester order); per group of 64 channels a = max|x'|,
s = fp16(min(a, 65504 * 7.5) / 7.5), code = clamp(floor(x' / s + 8), 0, 15) (8 when s = 0), level (c - 7.5) s.
"""

import numpy as np

from . import rotation

D = 128
TILE_BYTES = 2176
BLOCK_BYTES = 4 * TILE_BYTES
MAX_SCALE = 65504.0


def rope_angles(positions, rotary_dim, theta):
    i = np.arange(rotary_dim // 2, dtype=np.float64)
    return np.asarray(positions, dtype=np.float64)[:, None] * theta ** (-2.0 * i / rotary_dim)[None, :]


def rope(x, cos, sin, interleaved):
    """x [n, heads, 128]; cos, sin [n, rotary_dim / 2] (empty: no rotation)."""
    half = cos.shape[1]
    y = np.array(x, dtype=np.float64)
    a = slice(0, 2 * half, 2) if interleaved else slice(0, half)
    b = slice(1, 2 * half, 2) if interleaved else slice(half, 2 * half)
    c, s = cos[:, None, :], sin[:, None, :]
    y[..., a] = x[..., a] * c - x[..., b] * s
    y[..., b] = x[..., b] * c + x[..., a] * s
    return y


def to_rotated(x):
    return np.asarray(x, dtype=np.float64) @ rotation.hadamard(D)


def from_rotated(x):
    return np.asarray(x, dtype=np.float64) @ rotation.hadamard(D)  # H is symmetric and its own inverse


def quantise(xr):
    """Rotated rows [..., 128] -> codes uint8 [..., 128], scales float16 [..., 2], and x' / s + 8 (8 when s = 0)."""
    g = np.asarray(xr, dtype=np.float64).reshape(xr.shape[:-1] + (2, 64))
    s = (np.minimum(np.abs(g).max(-1), MAX_SCALE * 7.5) / 7.5).astype(np.float16)
    d = s.astype(np.float64)[..., None]
    t = np.where(d > 0, g / np.where(d > 0, d, 1.0) + 8.0, 8.0)
    return np.clip(np.floor(t), 0, 15).astype(np.uint8).reshape(xr.shape), s, t.reshape(xr.shape)


def levels(codes, scales):
    """Rotated-basis values of codes [..., 128] with scales [..., 2]."""
    g = codes.astype(np.float64).reshape(codes.shape[:-1] + (2, 64)) - 7.5
    return (g * scales.astype(np.float64)[..., None]).reshape(codes.shape)


def k_place(u, j):
    """(byte, nibble) of rotated channel j of token u (0..15) in a tile's K codes."""
    n = 4 * (j & 1) + 2 * ((j >> 2) & 1) + ((j >> 1) & 1)
    return 64 * u + 16 * ((j // 8) % 4) + 4 * (j // 32) + n // 2, n % 2


def v_place(u, j):
    """The same in a tile's V codes (which start at byte 1024)."""
    bit = lambda i: (j >> i) & 1  # noqa: E731
    lane = 4 * (j % 4 + 4 * bit(3)) + (u % 8) // 2
    return 1024 + 512 * bit(6) + 16 * lane + 4 * (bit(2) + 2 * bit(5)) + 2 * (u % 2) + u // 8, bit(4)


def unpack_block(block):
    """A block's bytes (uint8 [8704]) -> K codes, K scales, V codes, V scales of its 64 tokens."""
    kc, vc = np.zeros((64, D), np.uint8), np.zeros((64, D), np.uint8)
    ks, vs = np.zeros((64, 2), np.float16), np.zeros((64, 2), np.float16)
    u, j = np.meshgrid(np.arange(16), np.arange(D), indexing="ij")
    kb, kn = k_place(u, j)
    vb, vn = v_place(u, j)
    for t in range(4):
        tile = np.ascontiguousarray(block[t * TILE_BYTES:(t + 1) * TILE_BYTES])
        kc[16 * t:16 * t + 16] = (tile[kb] >> (4 * kn)) & 15
        vc[16 * t:16 * t + 16] = (tile[vb] >> (4 * vn)) & 15
        ks[16 * t:16 * t + 16] = tile[2048:2112].view(np.float16).reshape(16, 2)
        vs[16 * t:16 * t + 16] = tile[2112:2176].view(np.float16).reshape(16, 2)
    return kc, ks, vc, vs


def pack_block(kc, ks, vc, vs):
    """The inverse of unpack_block."""
    block = np.zeros(BLOCK_BYTES, np.uint8)
    for t in range(64):
        tile = block[(t // 16) * TILE_BYTES:(t // 16 + 1) * TILE_BYTES]
        for j in range(D):
            for code, (byte, nib) in ((kc[t, j], k_place(t % 16, j)), (vc[t, j], v_place(t % 16, j))):
                tile[byte] |= np.uint8(int(code) << (4 * nib))
        tile[2048 + 4 * (t % 16):2052 + 4 * (t % 16)] = ks[t].astype(np.float16).view(np.uint8)
        tile[2112 + 4 * (t % 16):2116 + 4 * (t % 16)] = vs[t].astype(np.float16).view(np.uint8)
    return block


def visible(p, n, window, sinks):
    """Truth values of positions 0..n-1: what the query at position p sees of a cache that holds n."""
    j = np.arange(n)
    v = j <= p
    if window >= 0:
        v &= (j < sinks) | (j > p - window)
    return v


def attend(q, k, v, p, window, sinks, sm_scale):
    """One query row q [128] at position p over k, v [n, 128]: (output, sum_j w_j |v_j|, largest sum_c |q_c k_jc| seen)."""
    see = visible(p, k.shape[0], window, sinks)
    if p < 0 or not see.any():
        return np.zeros(D), np.zeros(D), 0.0
    ks, vs = k[see], v[see]
    x = ks @ q * sm_scale
    w = np.exp(x - x.max())
    w /= w.sum()
    return w @ vs, w @ np.abs(vs), float((np.abs(ks) @ np.abs(q)).max())
