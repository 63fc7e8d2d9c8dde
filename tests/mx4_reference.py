"""4-bit floating point in 64 bits (numpy), for the tests of the CUDA operators.

Written from the formats' definitions alone: E2M1 codes with one scale to a
block of a row, E8M0 to 32 columns ("mxfp4") or E4M3 to 16 ("nvfp4", times one
number g for the matrix). Matrices are plain here: codes (rows, cols) and
scale bytes (rows, blocks); ``unpack`` reads the library's layout into that.
"""
import numpy as np

BLOCK = {"mxfp4": 32, "nvfp4": 16}
E2M1 = np.array([0, 0.5, 1, 1.5, 2, 3, 4, 6], dtype=np.float64)
MIDPOINTS = (E2M1[1:] + E2M1[:-1]) / 2


def blocks(cols, fmt):
    return -(-cols // BLOCK[fmt])


def e2m1(codes):
    codes = codes.astype(np.int64)
    return np.where(codes & 8, -1.0, 1.0) * E2M1[codes & 7]


def scale_value(b, fmt):
    b = b.astype(np.int64)
    if fmt == "mxfp4":
        return np.where(b == 255, np.nan, np.ldexp(1.0, b - 127))
    e, f = (b >> 3) & 15, b & 7
    v = np.where(e > 0, np.ldexp(1.0 + f / 8.0, e - 7), np.ldexp(f / 8.0, np.full_like(e, -6)))
    return np.where((b & 127) == 127, np.nan, v)


def round_e2m1(v):
    """Codes nearest to v: ties to the even code, magnitudes above 6 to 6."""
    a = np.abs(v)
    code = np.zeros(a.shape, dtype=np.int64)
    for i, mid in enumerate(MIDPOINTS):
        code += (a > mid) | ((a == mid) & (i % 2 == 1))
    return code | np.where(v < 0, 8, 0)


def round_e4m3(v):
    """E4M3 bytes nearest to v >= 0, at most 448."""
    table = scale_value(np.arange(127), "nvfp4")
    mids = (table[1:] + table[:-1]) / 2
    lo = np.searchsorted(mids, v, side="left")       # v == mids[lo]: a tie of lo and lo + 1
    tie = (lo < len(mids)) & (v == mids[np.minimum(lo, len(mids) - 1)])
    return lo + (tie & (lo % 2 == 1))


def tensor_scale(X):
    m = np.abs(X[np.isfinite(X)]).max(initial=0.0)
    g = 2.0 ** -100
    while 2688 * g < m and g < 2.0 ** 117:
        g *= 2
    return g


def quantize(X, fmt, g=1.0):
    """(codes, scale bytes) of X along its rows."""
    R, C = X.shape
    B, nb = BLOCK[fmt], blocks(C, fmt)
    x = np.zeros((R, nb * B))
    x[:, :C] = X
    x = x.reshape(R, nb, B)
    bad = ~np.isfinite(x).all(axis=2)
    m = np.where(bad, 0.0, np.abs(x).max(axis=2, initial=0.0))
    if fmt == "mxfp4":
        e = np.where(m > 0, np.frexp(np.where(m > 0, m, 1.0))[1] - 3, -127)
        s = np.where(bad, 255, np.clip(e, -127, 127) + 127)
    else:
        s = np.where(bad, 127, round_e4m3(m / (6 * g)))
    d = np.where(bad, 0.0, scale_value(np.where(bad, 0, s), fmt)) * g
    ok = (d > 0)[:, :, None]
    codes = round_e2m1(np.where(ok, np.where(ok, x, 0.0) / np.where(ok, d[:, :, None], 1.0), 0.0))
    return codes.reshape(R, nb * B)[:, :C], s


def values(codes, scales, fmt, g=1.0):
    C = codes.shape[1]
    return e2m1(codes) * np.repeat(scale_value(scales, fmt), BLOCK[fmt], axis=1)[:, :C] * g


def unpack(q):
    """(codes, scale bytes) of an Mx4Matrix, read from the documented layout,
    after checking that everything outside the matrix is zero."""
    R, C, fmt = q.rows, q.cols, q.fmt
    pitch = 16 * (-(-C // 32))
    raw = q.codes.cpu().numpy()[:R * pitch].reshape(R, pitch)
    both = np.stack((raw & 15, raw >> 4), axis=2).reshape(R, 2 * pitch)
    assert not both[:, C:].any(), "codes past the last column"
    tiles_k = -(-C // 256) * (256 // BLOCK[fmt] // 4)
    tiles_r = -(-R // 128)
    t = q.scales.cpu().numpy()[:tiles_r * tiles_k * 512].reshape(tiles_r, tiles_k, 32, 4, 4)
    flat = t.transpose(0, 3, 2, 1, 4).reshape(tiles_r * 128, tiles_k * 4)   # (r / 128, r % 128 / 32, r % 32)
    nb = blocks(C, fmt)
    assert not flat[R:].any() and not flat[:, nb:].any(), "scales outside the matrix"
    return both[:, :C], flat[:R, :nb]


def pack_codes(codes):
    """Row-major bytes of two codes, the lower column in the low half."""
    R, C = codes.shape
    c = np.zeros((R, C + C % 2), dtype=np.uint8)
    c[:, :C] = codes
    return np.ascontiguousarray(c[:, 0::2] | (c[:, 1::2] << 4))
