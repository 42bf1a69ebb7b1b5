"""The MXFP8 format and Philox in numpy's 64-bit types, for the checks of kernels that quantise: written from the
formats' definitions, without the library or its oracle."""
import numpy as np

E4M3 = np.array([(-1.0 if b & 128 else 1.0) * ((b & 7) * 2.0 ** -9 if (b >> 3) & 15 == 0
                                               else (8 + (b & 7)) * 2.0 ** (((b >> 3) & 15) - 10))
                 if b & 127 != 127 else np.nan for b in range(256)])


def decode(q, sc):
    """values of MXFP8 bytes q [..., C] with scales sc [..., ceil(C / 32)]"""
    s = np.ldexp(1.0, sc.astype(np.int64) - 127)
    return E4M3[q] * np.repeat(s, 32, axis=-1)[..., :q.shape[-1]]


def exponent(amax):
    """smallest e in [-127, 127] with amax <= 448 * 2^e; -127 for 0"""
    m, x = np.frexp(amax)
    return np.where(amax == 0, -127, np.clip(x - 9 + (m > 0.875), -127, 127)).astype(np.int64)


def blocks(v):
    """v [..., C] -> [..., ceil(C / 32), 32], the last block padded with zeros"""
    pad = -v.shape[-1] % 32
    v = np.concatenate([v, np.zeros(v.shape[:-1] + (pad,))], axis=-1) if pad else v
    return v.reshape(v.shape[:-1] + (-1, 32))


def check_rn(q, sc, v, rel, what=""):
    """q, sc: bytes of MXFP8 (round to nearest) of values that are within `rel` (relative) of the 64-bit v"""
    check_rn_abs(q, sc, v, rel * np.abs(v), what)


def check_rn_abs(q, sc, v, err, what=""):
    """q, sc: bytes of MXFP8 (round to nearest) of values that are within `err` (absolute, per element) of v.

    The scale must be the definition's, except where the block's largest value is within its error of a boundary
    between two scales; each element must be within half a step of its neighbourhood (2^-4 of the value, 2^-10 of the
    scale below E4M3's normal range) plus what `err` allows."""
    b, d = blocks(np.abs(v)), blocks(err)
    lo, hi = exponent(np.maximum(b - d, 0).max(-1)), exponent((b + d).max(-1))
    e = sc.astype(np.int64) - 127
    bad = (e < lo) | (e > hi)
    assert not bad.any(), "%s: %d scales off" % (what, bad.sum())
    step = np.maximum(np.abs(v) * 2.0 ** -4, np.repeat(np.ldexp(1.0, e - 10), 32, axis=-1)[..., :v.shape[-1]])
    over = np.abs(decode(q, sc) - v) - step - 2 * err
    assert over.max(initial=-1.0) <= 0, "%s: %d of %d elements beyond half a step" % (what, (over > 0).sum(), v.size)


def philox(counter, key):
    """Philox4x32-10 (Salmon et al., SC'11) of four uint64 arrays that hold 32-bit words"""
    c = [np.asarray(x, np.uint64) for x in counter]
    k0, k1 = np.uint64(key & 0xFFFFFFFF), np.uint64(key >> 32)
    low, sh = np.uint64(0xFFFFFFFF), np.uint64(32)
    for _ in range(10):
        a, b = c[0] * np.uint64(0xD2511F53), c[2] * np.uint64(0xCD9E8D57)
        c = [(b >> sh) ^ c[1] ^ k0, b & low, (a >> sh) ^ c[3] ^ k1, a & low]
        k0, k1 = (k0 + np.uint64(0x9E3779B9)) & low, (k1 + np.uint64(0xBB67AE85)) & low
    return c


def random_bits(n, seed, tag, word3):
    """the 16 bits of each of n elements: see pmn_requant_transpose_sr_mxfp8"""
    j = np.arange((n + 15) // 16, dtype=np.uint64)
    w = np.stack(philox([j & np.uint64(0xFFFFFFFF), j >> np.uint64(32), np.full_like(j, tag), np.full_like(j, word3)], seed), 1)
    lo, hi = w & np.uint64(0xFFFF), w >> np.uint64(16)
    rev = np.array([int("{:016b}".format(i)[::-1], 2) for i in range(65536)], np.uint64)
    return np.stack([lo, rev[lo.astype(np.int64)], hi, rev[hi.astype(np.int64)]], 2).reshape(-1)[:n].astype(np.int64)
