"""MXFP4 in exact arithmetic, for the tests: numpy in 64 bits."""
import numpy as np

LEVELS = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])


def quantize(x):
    """(codes, scales, values) of x [..., k], float64 holding bf16 or binary32 values."""
    v = np.asarray(x, np.float64)
    v = v.reshape(v.shape[:-1] + (-1, 32))
    with np.errstate(invalid="ignore"):
        m = np.abs(v).max(-1, keepdims=True)
    finite = np.isfinite(m)
    m = np.where(finite, m, 0.0)
    X = np.where(m > 0, np.frexp(m)[1] - 1 - 2, -127)   # frexp: m = f 2^e with f in [1/2, 1)
    X = np.maximum(X, -127)
    y = np.ldexp(np.abs(np.where(finite, v, 0.0)), -X)
    below = np.clip(np.searchsorted(LEVELS, y, side="right") - 1, 0, 6)
    down, up = y - LEVELS[below], LEVELS[below + 1] - y
    code = np.where((up < down) | ((up == down) & (below % 2 == 1)), below + 1, below)
    sign = np.signbit(v) & finite
    values = np.where(finite, np.where(sign, -1.0, 1.0) * np.ldexp(LEVELS[code], X), np.nan)
    code = np.where(finite, code | (sign.astype(np.int64) << 3), 0)
    scales = np.where(finite, X + 127, 255)[..., 0].astype(np.uint8)
    code = code.reshape(code.shape[:-2] + (-1,)).astype(np.uint8)
    return code[..., 0::2] | (code[..., 1::2] << 4), scales, values.reshape(np.shape(x))


def decode(codes, scales):
    """What codes and scales stand for; NaN under scale 255."""
    lv = np.concatenate([LEVELS, -LEVELS])
    v = np.stack([lv[codes & 15], lv[codes >> 4]], -1).reshape(codes.shape[:-1] + (-1, 32))
    s = scales.astype(np.int64)[..., None]
    return np.where(s == 255, np.nan, np.ldexp(v, s - 127)).reshape(codes.shape[:-1] + (-1,))
