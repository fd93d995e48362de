"""The microscaled storage from its definition, in numpy (include/gemm.h,
gemm_mx_format_t): what a stored matrix holds, and its 64-bit values.  Shares
no code with the library."""
import numpy as np

BLOCK = {"fp4": 32, "fp4_e4m3": 16, "int8": 32}
E2M1 = np.array([0, 0.5, 1, 1.5, 2, 3, 4, 6], dtype=np.float64)


def _e4m3_table():
    t = np.empty(128, dtype=np.float64)
    for b in range(128):
        e, m = b >> 3, b & 7
        t[b] = m / 8 * 2.0 ** -6 if e == 0 else (1 + m / 8) * 2.0 ** (e - 7)
    t[127] = np.nan
    return t


E4M3 = _e4m3_table()


def nearest(y, table):
    """Place in the ascending `table` nearest to y >= 0, ties to the even place."""
    hi = np.clip(np.searchsorted(table, y), 0, len(table) - 1)
    lo = np.maximum(hi - 1, 0)
    dl, dh = y - table[lo], table[hi] - y
    take_lo = (dl < dh) | ((dl == dh) & (lo % 2 == 0))
    return np.where((hi > 0) & take_lo, lo, hi)


def row_bytes(fmt, cols):
    b = cols if fmt == "int8" else -(-cols // 2)
    return -(-b // 16) * 16


def scale_place(r, b, tiles):
    return ((r // 128) * tiles + b // 4) * 512 + r % 32 * 16 + r % 128 // 32 * 4 + b % 4


def scale_values(byte, fmt):
    byte = np.asarray(byte).astype(np.int64)
    if fmt == "fp4_e4m3":
        return E4M3[byte]
    return np.where(byte == 255, np.nan, 2.0 ** (np.minimum(byte, 254) - 127.0))


def store(x, fmt, mult=1.0):
    """(codes uint8 [rows, row_bytes], scale tiles uint8, values float64) of the
    float32-valued matrix x."""
    rows, cols = x.shape
    t = (x.astype(np.float32) * np.float32(mult)).astype(np.float32)
    b = BLOCK[fmt]
    nb = -(-cols // b)
    p = np.zeros((rows, nb * b), dtype=np.float32)
    p[:, :cols] = t
    p = p.reshape(rows, nb, b)
    with np.errstate(all="ignore"):
        amax = np.abs(p).max(axis=2)
        bad = ~np.isfinite(p).all(axis=2)
        amax = np.where(bad, 0, amax).astype(np.float32)
        if fmt == "fp4_e4m3":
            want = (amax / np.float32(6)).astype(np.float32)
            byte = nearest(want.astype(np.float64), E4M3[:127])
            s = E4M3[byte]
            y = np.where(s[:, :, None] > 0,
                         (p / s.astype(np.float32)[:, :, None]).astype(np.float64), 0.0)
            byte = np.where(bad, 0x7F, byte)
        else:
            e = np.frexp(amax.astype(np.float64))[1] - 1 - (2 if fmt == "fp4" else 6)
            e = np.where(amax > 0, np.maximum(e, -127), -127)
            y = p.astype(np.float64) * 2.0 ** -e.astype(np.float64)[:, :, None]
            byte = np.where(bad, 255, e + 127)
        y = np.where(bad[:, :, None], 0.0, y)
        neg = np.signbit(p) & ~bad[:, :, None]
    scale = scale_values(byte, fmt)
    if fmt == "int8":
        code = np.clip(np.rint(y), -127, 127)
        value = code * scale[:, :, None]
        raw = code.astype(np.int8).view(np.uint8).reshape(rows, -1)[:, :cols]
    else:
        idx = nearest(np.abs(y), E2M1)
        value = np.where(neg, -E2M1[idx], E2M1[idx]) * scale[:, :, None]
        nib = (idx | (neg.astype(np.int64) << 3)).astype(np.uint8).reshape(rows, -1)[:, :cols]
        nib = np.pad(nib, ((0, 0), (0, cols % 2)))
        raw = nib[:, 0::2] | (nib[:, 1::2] << 4)
    codes = np.zeros((rows, row_bytes(fmt, cols)), dtype=np.uint8)
    codes[:, :raw.shape[1]] = raw
    tiles = -(-nb // 4)
    st = np.zeros(-(-rows // 128) * tiles * 512, dtype=np.uint8)
    r, k = np.meshgrid(np.arange(rows), np.arange(nb), indexing="ij")
    st[scale_place(r, k, tiles)] = byte
    return codes, st, value.reshape(rows, -1)[:, :cols]


def load(codes, st, rows, cols, fmt):
    """float64 values of a stored matrix."""
    b = BLOCK[fmt]
    tiles = -(-(-(-cols // b)) // 4)
    r, c = np.meshgrid(np.arange(rows), np.arange(cols), indexing="ij")
    scale = scale_values(st[scale_place(r, c // b, tiles)], fmt)
    if fmt == "int8":
        return codes[:, :cols].view(np.int8).astype(np.float64) * scale
    nib = (codes[r, c // 2] >> (4 * (c % 2))) & 15
    v = E2M1[nib & 7]
    return np.where(nib > 7, -v, v) * scale


def gelu(x):
    import math
    erfc = np.vectorize(math.erfc, otypes=[np.float64])
    return x * 0.5 * erfc(-x / math.sqrt(2.0))


def slope(x, act):
    import math
    if act == "relu":
        return (x > 0).astype(np.float64)
    if act == "gelu":
        erfc = np.vectorize(math.erfc, otypes=[np.float64])
        return 0.5 * erfc(-x / math.sqrt(2.0)) + x * np.exp(-x * x / 2) / math.sqrt(2 * math.pi)
    return np.ones_like(x)
