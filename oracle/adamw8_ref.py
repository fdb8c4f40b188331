"""numpy reference of AdamW on 8-bit moments.  The codes are defined by fp32
arithmetic with every operation rounded by itself, so the moments are computed
in numpy's float32, one operation at a time, and the codes in integers; the
weights are computed in fp64 from the moments.  Shares no code with the library.
"""
from __future__ import annotations

import numpy as np

BLOCK = 256
TOP = (127, 255)  # largest code of the first and second moment
M32 = 0xFFFFFFFF


def mix(x):
    x = int(x) & M32
    x ^= x >> 16
    x = x * 0x6A09E667 & M32
    x ^= x >> 15
    x = x * 0xBB67AE85 & M32
    return x ^ (x >> 16)


def random_bits(numel, step, moment, first=0):
    """16 random bits of elements first .. first + numel - 1."""
    step &= (1 << 64) - 1
    key = mix((step & M32) ^ mix(step >> 32))
    i = np.arange(first, first + numel, dtype=object)
    out = np.empty(numel, dtype=np.int64)
    for j, el in enumerate(i):
        q = int(el) // 4
        h = mix((q & M32) ^ ((q >> 32) * 0x9E3779B1 & M32) ^ key)
        turn = 8 * (int(el) % 4)
        h = ((h >> turn) | (h << (32 - turn))) & M32
        out[j] = (h >> 16) if moment else (h & 0xFFFF)
    return out


def bits(x):
    """Bits of |x|, NaN as 0x7fc00000."""
    x = np.asarray(x, dtype=np.float32)
    return np.where(np.isnan(x), 0x7FC00000, x.view(np.uint32) & 0x7FFFFFFF).astype(np.int64)


def from_bits(u):
    return np.asarray(u, dtype=np.int64).astype(np.uint32).view(np.float32)


def encode(x, step, moment, rand=None):
    """(codes uint8, offsets) of a flat fp32 array; the last block may be short."""
    x = np.asarray(x, dtype=np.float32).reshape(-1)
    n = x.size
    r = random_bits(n, step, moment) if rand is None else rand
    u = bits(x)
    codes, offs = np.zeros(n, dtype=np.uint8), []
    for a in range(0, n, BLOCK):
        b = min(n, a + BLOCK)
        top = -(-int(u[a:b].max()) // (1 << 20))
        off = max(0, top - TOP[moment])
        lo = from_bits((off + 1) << 20)
        k = (u[a:b] + 16 * r[a:b]) // (1 << 20) - off
        if moment:
            small = (u[a:b] > 0).astype(np.int64)
        else:
            share = ((r[a:b] + 0.5) / 65536.0).astype(np.float32)  # 17 bits: exact
            small = (np.abs(x[a:b]) > lo * share).astype(np.int64)
        k = np.where(u[a:b] < (off + 1) << 20, small, k)
        assert k.min() >= 0 and k.max() <= TOP[moment]
        sign = 0 if moment else np.where(np.signbit(x[a:b]), 128, 0)
        codes[a:b] = k + sign
        offs.append(off)
    return codes, np.array(offs, dtype=np.uint16)


def decode(codes, offs, moment):
    """fp32 values of codes."""
    c = np.asarray(codes, dtype=np.int64)
    off = np.repeat(np.asarray(offs, dtype=np.int64), BLOCK)[:c.size]
    k = c if moment else c & 127
    x = from_bits(np.where(k > 0, (k + off) << 20, 0)).copy()
    return x if moment else np.where(c >= 128, -x, x)


def state_bytes(numel):
    nb = -(-numel // BLOCK)
    return nb * BLOCK + -(-2 * nb // 16) * 16


def to_state(codes, offs, fill=0):
    """The buffer of a moment; what lies behind the codes and offsets is `fill`."""
    n, nb = codes.size, offs.size
    s = np.full(state_bytes(n), fill, dtype=np.uint8)
    s[:n] = codes
    s[nb * BLOCK:nb * BLOCK + 2 * nb] = offs.view(np.uint8)
    return s


def from_state(state, numel):
    nb = -(-numel // BLOCK)
    return state[:numel], state[nb * BLOCK:nb * BLOCK + 2 * nb].view(np.uint16)


def moments(g, m, v, beta1, beta2):
    """The new moments in fp32, each operation rounded by itself."""
    f = np.float32
    g, m, v = (np.asarray(t, dtype=f) for t in (g, m, v))
    c1, c2 = f(1) - f(beta1), f(1) - f(beta2)
    with np.errstate(all="ignore"):
        m = m + (g - m) * c1
        v = v + (g * g - v) * c2
    return m, v


def weights(w, m, v, lr, beta1, beta2, eps, wd, t):
    """The new weights in fp64 from the new moments."""
    f = lambda x: float(np.float32(x))
    w, m, v = (np.asarray(x, dtype=np.float64) for x in (w, m, v))
    step = f(lr) * np.sqrt(1 - f(beta2) ** t) / (1 - f(beta1) ** t)
    with np.errstate(all="ignore"):
        return w * (1 - f(lr) * f(wd)) - step * m / (f(eps) + np.sqrt(v))
