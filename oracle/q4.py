"""Oracle: matrices of 4-bit integers with a BF16 scale (and a zero point) per
group of columns, in fp64 (test infrastructure only).

value[n, k] = scale[n, k // group] * (q[n, k] - zero[n, k // group]), q in
0..15, zero 8 without zero points.  ``layout`` places codes, scales and zero
points element by element at the byte (and nibble) the block's definition
names; ``parse`` is its inverse, written from the same definition.

Pins (tests/test_oracle_q4.py): layout and parse invert each other at sizes
off the tile; every code lands in a place of its own; encode is within half a
step of the input and reproduces values on the grid.
"""

import numpy as np

from . import formats


def _tiles(N, K):
    return (N + 15) // 16, (K + 127) // 128


def sections(N, K, group, zero):
    """(codes, scales, zero points, total) bytes of a block."""
    t, b = _tiles(N, K)
    g = b * (128 // group)
    sizes = (t * b * 1024, t * g * 32, t * g * 16 if zero else 0)
    return sizes + (sum(sizes),)


def _places(N, K):
    """byte offset and nibble of every element of a matrix"""
    _, b = _tiles(N, K)
    n, k = np.meshgrid(np.arange(N), np.arange(K), indexing="ij")
    lane = 16 * ((k % 32) // 8) + n % 16
    tile = (n // 16) * b + k // 128
    dword = (k % 128) // 32
    i = k % 8
    nibble = i // 2 + 4 * (i % 2)
    return tile * 1024 + lane * 16 + dword * 4 + nibble // 2, nibble % 2


def layout(q, scale_bits, zeros, group):
    """Block bytes of codes q [N, K], BF16 scale bits [N, G], zeros [N, G] or None."""
    N, K = q.shape
    t, b = _tiles(N, K)
    nc, ns, nz, total = sections(N, K, group, zeros is not None)
    out = np.zeros(total, dtype=np.uint8)
    pad = np.full((16 * t, 128 * b), 8, dtype=np.uint8)
    pad[:N, :K] = q
    at, high = _places(16 * t, 128 * b)
    np.bitwise_or.at(out, at.ravel(), (pad << (4 * high)).astype(np.uint8).ravel())
    G = b * (128 // group)
    s = np.zeros((16 * t, G), dtype=np.uint16)
    s[:N, :scale_bits.shape[1]] = scale_bits
    out[nc:nc + ns] = s.reshape(t, 16, G).transpose(0, 2, 1).copy().view(np.uint8).ravel()
    if zeros is not None:
        z = np.full((16 * t, G), 8, dtype=np.uint8)
        z[:N, :zeros.shape[1]] = zeros
        out[nc + ns:] = z.reshape(t, 16, G).transpose(0, 2, 1).ravel()
    return out


def parse(block, N, K, group, zero):
    """(q [N, K], scale bits [N, ceil(K / group)], zeros or None) of a block."""
    t, b = _tiles(N, K)
    nc, ns, nz, _ = sections(N, K, group, zero)
    at, high = _places(N, K)
    q = (block[at] >> (4 * high)) & 15
    G = b * (128 // group)
    used = (K + group - 1) // group
    untile = lambda v: v.reshape(t, G, 16).transpose(0, 2, 1).reshape(16 * t, G)[:N, :used]
    s = untile(block[nc:nc + ns].copy().view(np.uint16))
    z = untile(block[nc + ns:nc + ns + nz]) if zero else None
    return q.astype(np.uint8), s, z


def decode(q, scale_bits, zeros, group):
    """fp64 values."""
    N, K = q.shape
    s = np.repeat(formats.bf16_decode(scale_bits), group, axis=1)[:, :K]
    z = 8.0 if zeros is None else np.repeat(zeros.astype(np.float64), group, axis=1)[:, :K]
    return (q.astype(np.float64) - z) * s


def encode(v, group, zero):
    """Quantise values [N, K] with the fp32 steps of the encoder's definition.
    Returns (q, scale bits, zeros or None)."""
    v = np.asarray(v, dtype=np.float32)
    N, K = v.shape
    G = (K + group - 1) // group
    pad = np.zeros((N, G * group), dtype=np.float32)
    pad[:, :K] = v
    p = pad.reshape(N, G, group)
    lo = np.minimum(p.min(axis=2), np.float32(0))
    hi = np.maximum(p.max(axis=2), np.float32(0))
    s = (hi - lo) / np.float32(15) if zero else np.maximum(hi, -lo) / np.float32(7)
    bits = formats.bf16_round(s.astype(np.float32))
    sr = formats.bf16_decode(bits).astype(np.float32)
    safe = np.where(sr > 0, sr, np.float32(1)).astype(np.float32)
    z = np.where(sr > 0, np.clip(np.rint(-lo / safe), 0, 15), 8).astype(np.float32) if zero \
        else np.full_like(sr, 8)
    q = np.clip(np.rint((p / safe[..., None]).astype(np.float32)) + z[..., None], 0, 15)
    q = np.where(sr[..., None] > 0, q, z[..., None])
    q = q.reshape(N, -1)[:, :K].astype(np.uint8)
    return q, bits, z.astype(np.uint8) if zero else None
