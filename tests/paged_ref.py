"""Plain numpy forms of the paged cache for its tests: a rotation and a
quantisation in float32, operation by operation as the call defines them, and
everything again in float64; the attention of one query in float64."""
import numpy as np

LEVEL = {"int8": 127.0, "e4m3": 448.0}
F32 = np.float32


def rotate(x, t, interleaved, back=False):
    """x [..., d] turned by table rows t [..., rot], in x's own type."""
    rot = t.shape[-1]
    h = rot // 2
    y = x.copy()
    if rot == 0:
        return y
    c, s = t[..., :h].astype(x.dtype), t[..., h:].astype(x.dtype)
    if back:
        s = -s
    a, b = (slice(0, rot, 2), slice(1, rot, 2)) if interleaved else (slice(0, h), slice(h, rot))
    y[..., a] = x[..., a] * c - x[..., b] * s
    y[..., b] = x[..., b] * c + x[..., a] * s
    return y


def e4m3_values():
    """The 256 values of the e4m3 codes."""
    v = np.zeros(256)
    for code in range(256):
        e, m = (code >> 3) & 15, code & 7
        x = m * 2.0 ** -9 if e == 0 else (8 + m) * 2.0 ** (e - 10)
        if e == 15 and m == 7:
            x = np.nan
        v[code] = -x if code & 128 else x
    return v


E4M3 = e4m3_values()
_POS = E4M3[:127]


def e4m3_code(x):
    """Codes of float32 values by nearest even, |x| <= 448 (1 + 2^-22)."""
    a = np.abs(x).astype(np.float64)
    hi = np.clip(np.searchsorted(_POS, a), 1, 126)
    lo = hi - 1
    mid = 0.5 * (_POS[lo] + _POS[hi])
    code = np.where((a > mid) | ((a == mid) & (hi % 2 == 0)), hi, lo)
    return (code | np.where(np.signbit(x), 128, 0)).astype(np.uint8)


def quantise(x, cache):
    """Codes (uint8 bits) and scales of groups x [n, 8, d] float32, each
    operation rounded to float32."""
    top = F32(LEVEL[cache])
    with np.errstate(invalid="ignore", over="ignore"):
        a = np.abs(x).max((1, 2))
        fine = np.isfinite(a)
        safe = np.maximum(np.where(fine, a, F32(1)), top * F32(2.0 ** -126))
        f = (F32(1) / safe) * top
        y = np.where(fine[:, None, None], x * f[:, None, None], F32(0))
    code = np.rint(y).astype(np.int8).view(np.uint8) if cache == "int8" else e4m3_code(y)
    return code, np.where(fine, safe / top, F32(np.nan))


def held(code, scale, cache):
    """The float64 values of codes [..., 8, d] (uint8 bits) with scales [...]."""
    v = code.view(np.int8).astype(np.float64) if cache == "int8" else E4M3[code]
    return v * scale.astype(np.float64)[..., None, None]


def attend(q, k, v, scale):
    """O and lse of q [G, d] over k, v [n, d] in float64."""
    s = scale * (q @ k.T)
    m = s.max(1, keepdims=True)
    w = np.exp(s - m)
    l = w.sum(1, keepdims=True)
    return (w / l) @ v, (m + np.log(l))[:, 0]


def top(scores, k):
    """Ascending indices of the k highest, equal scores to the lower index."""
    return np.sort(np.argsort(-scores, kind="stable")[:k])
