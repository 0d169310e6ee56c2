"""q4_0 block quantisation of a paged pool, written out from the definition.

32 consecutive values along head_dim share one fp16 scale and have a code of four bits each:
    m    = the block's value of greatest magnitude; of +a and -a the negative one
    q_i  = min(round(-8 x_i / m), 7)   the exact quotient, ties away from zero: a code in [-8, 7]
    d_h  = fp16(-m / 8)                round to nearest even, subnormals kept
An all-zero block has codes of zero and d_h = +0.  The stored value is d_h * q_i.

The quotient of two float32 values, as a float64, rounds as the exact one does: where it is not a
tie it is at least 2^-28 away from one.

Packing: a block's 16 bytes are four little-endian 32-bit words; value i of a word's eight lies, as
q + 8, in the four bits from bit 16 (i % 2) + 4 (i // 2).
"""

import numpy as np

BLOCK = 32
_SHIFT = np.array([16 * (i % 2) + 4 * (i // 2) for i in range(8)], dtype=np.uint32)


def quantize_blocks(x):
    """(d_h float16 [..., n/32], q int8 [..., n]) of float32 values [..., n], n a multiple of 32."""
    x = np.asarray(x, dtype=np.float32)
    if not np.isfinite(x).all():
        raise ValueError("q4_0 quantisation is defined for finite inputs only")
    if x.shape[-1] % BLOCK:
        raise ValueError("last axis must be a multiple of 32")
    b = x.astype(np.float64).reshape(x.shape[:-1] + (x.shape[-1] // BLOCK, BLOCK))
    top, low = b.max(axis=-1), b.min(axis=-1)
    m = np.where(top > -low, top, low)
    some = m != 0
    y = -8.0 * b / np.where(some, m, 1.0)[..., None]
    q = np.minimum(np.copysign(np.floor(np.abs(y) + 0.5), y), 7)
    q = np.where(some[..., None], q, 0).astype(np.int8).reshape(x.shape)
    d = np.where(some, m / -8.0, 0.0).astype(np.float16)
    return d, q


def pack(q):
    """The bytes (uint8 [..., n/2]) of codes [..., n]."""
    u = (np.asarray(q).astype(np.int32) + 8).astype(np.uint32).reshape(q.shape[:-1] + (q.shape[-1] // 8, 8))
    return np.ascontiguousarray((u << _SHIFT).sum(-1).astype("<u4")).view(np.uint8)


def unpack(b):
    """The codes (int8 [..., 2 n]) of bytes [..., n]."""
    w = np.ascontiguousarray(b).view("<u4")
    q = (w[..., None] >> _SHIFT) & 15
    return (q.astype(np.int8) - 8).reshape(b.shape[:-1] + (b.shape[-1] * 2,))


def dequantize_blocks(d_h, q):
    """float32 values d_h * q, exact."""
    q = np.asarray(q)
    qb = q.reshape(q.shape[:-1] + (q.shape[-1] // BLOCK, BLOCK)).astype(np.float32)
    return (np.asarray(d_h).astype(np.float32)[..., None] * qb).reshape(q.shape)
