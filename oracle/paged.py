"""fp64 oracle of the paged 8-bit cache: codes and scales, rotation, append, attention.

Written from the definitions in numpy; shares no code with the CUDA path (test infrastructure only).
"""

from __future__ import annotations

import numpy as np

QMAX = {"e4m3": 448.0, "int8": 127.0}


def e4m3_values() -> np.ndarray:
    """The value of each of the 256 codes (sign, 4 exponent bits with bias 7, 3 mantissa bits; S.1111.111 is NaN)."""
    c = np.arange(256)
    e, m = (c >> 3) & 15, c & 7
    v = np.where(e == 0, m * 2.0 ** -9, (8 + m) * 2.0 ** (e - 10.0))
    v[(c & 127) == 127] = np.nan
    return np.where(c >= 128, -v, v)


def values(codes: np.ndarray, kind: str) -> np.ndarray:
    """Codes (uint8 bytes) as fp64, without their scale."""
    return codes.view(np.int8).astype(np.float64) if kind == "int8" else e4m3_values()[codes]


def encode(y: np.ndarray, kind: str) -> np.ndarray:
    """The bytes nearest to y (already divided by the scale): ties to even, saturating, NaN as 0."""
    y = np.where(np.isnan(y), 0.0, np.clip(y, -QMAX[kind], QMAX[kind]))
    if kind == "int8":
        return np.rint(y).astype(np.int8).view(np.uint8)
    mag = np.abs(y)
    step = 2.0 ** np.maximum(np.floor(np.log2(np.maximum(mag, 2.0 ** -30))) - 3, -9)
    mag = np.rint(mag / step) * step
    table = e4m3_values()[:127]
    return (np.searchsorted(table, mag) | np.where(np.signbit(y), 128, 0)).astype(np.uint8)


def scale_for(amax: float, kind: str) -> float:
    if kind == "int8":
        return max(float(np.float32(amax) * (np.float32(1) / np.float32(127))), 2.0 ** -126)
    x = -126
    while 448.0 * 2.0 ** x < amax:
        x += 1
    return 2.0 ** x


def rotate(x: np.ndarray, table: np.ndarray, pos: np.ndarray, interleaved: bool) -> np.ndarray:
    """x [n, heads, d] in fp64, table [positions, rot]: cosines then sines."""
    rot = table.shape[1]
    r = rot // 2
    a = np.arange(0, rot, 2) if interleaved else np.arange(r)
    b = a + 1 if interleaved else a + r
    cos, sin = table[pos, None, :r].astype(np.float64), table[pos, None, r:].astype(np.float64)
    y = x.copy()
    y[..., a] = x[..., a] * cos - x[..., b] * sin
    y[..., b] = x[..., b] * cos + x[..., a] * sin
    return y


def append(codes, scales, x, start: int, pages, kind: str, page: int) -> None:
    """x [n, heads, d] (fp32 values) go to positions start .. of a sequence in place: codes [pages, heads, page, d] bytes,
    scales [pages, heads] fp32; pages: the sequence's table row (entries outside the cache are skipped)."""
    n = x.shape[0]
    for lo in range(start // page * page, start + n, page):
        pid = int(pages[lo // page])
        if not 0 <= pid < codes.shape[0]:
            continue
        a, z = max(lo, start), min(lo + page, start + n)
        part = x[a - start:z - start]
        for h in range(x.shape[1]):
            y = part[:, h]
            fine = np.abs(y[np.isfinite(y)])
            want = scale_for(float(fine.max()) if fine.size else 0.0, kind)
            now = want
            if a > lo:
                was = float(scales[pid, h])
                now = was if was >= want else want
                if now != was:
                    ratio = np.float32(was) * (np.float32(1) / np.float32(now))
                    old = values(codes[pid, h, :a - lo], kind).astype(np.float32)
                    codes[pid, h, :a - lo] = encode((old * ratio).astype(np.float64), kind)
            scales[pid, h] = np.float32(now)
            inv = np.float32(1) / np.float32(now)
            with np.errstate(invalid="ignore", over="ignore"):
                codes[pid, h, a - lo:z - lo] = encode((y.astype(np.float32) * inv).astype(np.float64), kind)


def attend(q, K, V, n_new: int, kv_len: int, scale: float, window: int = 0, n_sink: int = 0, gone=None):
    """q [n_new, heads, d], K, V [kv_len, kv_heads, d] fp64 (the sequence's values); `gone` marks tokens that are not
    there.  Returns out, lse, and for tolerances sum p |v| and the largest sum |q| |k| scale of a visible token."""
    G = q.shape[1] // K.shape[1]
    out, most = np.zeros_like(q), np.zeros(q.shape[:2])
    lse, mag = np.full(q.shape[:2], -np.inf), np.zeros_like(q)
    j = np.arange(kv_len)
    for i in range(n_new):
        t = kv_len - n_new + i
        seen = j <= t
        if window:
            seen &= (j > t - window) | (j < n_sink)
        if gone is not None:
            seen &= ~gone
        if not seen.any():
            continue
        for u in range(q.shape[1]):
            k, v = K[seen, u // G], V[seen, u // G]
            z = k @ q[i, u] * scale
            m = z.max()
            p = np.exp(z - m)
            lse[i, u] = m + np.log(p.sum())
            p /= p.sum()
            out[i, u], mag[i, u] = p @ v, p @ np.abs(v)
            most[i, u] = (np.abs(k) @ np.abs(q[i, u])).max() * scale
    return out, lse, mag, most
