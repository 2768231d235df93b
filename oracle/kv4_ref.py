"""The 4-bit cache rows in 64 bits, from their definition (include/hpc_decode.h, hpc_rope_kv4_write):
72 bytes a row, 64 of e2m1 codes and 8 of e4m3 scales of sixteen elements each. Test infrastructure."""
import numpy as np

E2M1 = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])


def _e4m3():
    """The 127 values of the codes 0 .. 126, from sign, four bits of exponent (bias 7), three of mantissa."""
    c = np.arange(127)
    e, m = c >> 3, c & 7
    return np.where(e == 0, m / 8.0 * 2.0 ** -6, (1 + m / 8.0) * 2.0 ** (e - 7.0))


E4M3 = _e4m3()


def nearest(x, table):
    """Index of the table's nearest value to each x >= 0: ties to the even index, saturating; NaN gives -1."""
    mids = (table[1:] + table[:-1]) / 2
    x = np.asarray(x, np.float64)
    low, high = np.searchsorted(mids, x, "left"), np.searchsorted(mids, x, "right")
    return np.where(np.isnan(x), -1, np.where(low % 2 == 0, low, high))  # (they differ at a midpoint only)


def units(scale_codes, ts):
    """fl(scale * ts) in fp32, NaN of a scale of code 127."""
    s = np.where(scale_codes == 127, np.nan, E4M3[np.minimum(scale_codes, 126)])
    return (s.astype(np.float32) * np.float32(ts)).astype(np.float64)


def scales(x, ts):
    """Scale codes of x [..., 128] float64."""
    a = np.abs(x).reshape(x.shape[:-1] + (8, 16)).max(-1)  # (NaN where one of them is)
    with np.errstate(over="ignore"):
        c = nearest(a / np.float64(np.float32(6) * np.float32(ts)), E4M3)
    return np.where(c < 0, 127, c)


def codes(x, scale_codes, ts):
    """e2m1 codes (sign in bit 3) of x [..., 128] over given scales; 0 where the scale is 0 or NaN."""
    u = np.repeat(units(scale_codes, ts), 16, -1)
    ok = u > 0
    with np.errstate(over="ignore", invalid="ignore"):
        c = nearest(np.where(ok, np.abs(x) / np.where(ok, u, 1.0), 0.0), E2M1)
    return np.where(ok, c | (np.signbit(x) << 3), 0)


def rows(x, ts):
    """x [..., 128] float64 to uint8 [..., 72]."""
    s = scales(x, ts)
    c = codes(x, s, ts)
    return np.concatenate([c[..., 0::2] | (c[..., 1::2] << 4), s], -1).astype(np.uint8)


def split(r):
    """(code values [..., 128], scale codes [..., 8]) of rows."""
    n = np.stack([r[..., :64] & 15, r[..., :64] >> 4], -1).reshape(r.shape[:-1] + (128,))
    return np.where(n >= 8, -1.0, 1.0) * E2M1[n & 7], r[..., 64:].astype(np.int64)


def values(r, ts):
    """What rows stand for, in float64."""
    c, s = split(r)
    s = np.where((s & 127) == 127, np.nan, np.where(s >= 128, -1.0, 1.0) * E4M3[np.minimum(s & 127, 126)])
    return c * np.repeat(s, 16, -1) * np.float64(np.float32(ts))
