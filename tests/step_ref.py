"""Plain references, in 64 bits on the CPU, of the operators around the attention of recent tokens, and how far their
results may be from them. Written from the contracts in include/c128compress.h."""
import math

import numpy as np

HEAD, NOPE, ROPE = 512, 448, 64
HALF = {"bf16": 2.0 ** -8, "fp32": 2.0 ** -24}   # half a step, relative to the value


def steps(theta=10000.0, scaling="none", factor=1.0, original_positions=65536, beta_fast=32.0, beta_slow=1.0, magnitude=1.0,
          width=64):
    """Radians per position of each pair."""
    out = []
    for i in range(width // 2):
        f = theta ** (-2 * i / width)
        if scaling == "linear":
            f /= factor
        if scaling == "yarn":
            low, high = (width * math.log(original_positions / (2 * math.pi * b)) / (2 * math.log(theta))
                         for b in (beta_fast, beta_slow))
            low, high = max(math.floor(low), 0), min(math.ceil(high), width - 1)
            g = min(max((i - low) / max(high - low, 0.001), 0.0), 1.0)
            f = f * (1 - g) + f / factor * g
        out.append(f)
    return np.array(out)


def cos_sin(first, rows, magnitude=1.0, **rope):
    """(table [rows, width], its tolerance)."""
    turns = (first + np.arange(rows, dtype=np.float64))[:, None] * (steps(magnitude=magnitude, **rope) / (2 * math.pi))
    angle = 2 * math.pi * (turns - np.floor(turns))
    off = abs(magnitude) * (2.0 ** -30 + 2.0 ** -48 * turns)
    c, s = np.cos(angle) * magnitude, np.sin(angle) * magnitude
    # (the reference's own angle is off by as much as the steps' rounding again)
    return np.concatenate([c, s], 1), np.concatenate([2 * off + 2.0 ** -22 * np.abs(c), 2 * off + 2.0 ** -22 * np.abs(s)], 1)


def rotate(x, cs, first, layout, inverse):
    """(x with the columns behind `first` turned, magnitude of the sums): x [T, H, D], cs [T, R] of each token."""
    half = cs.shape[1] // 2
    c, s = cs[:, None, :half], cs[:, None, half:] * (-1 if inverse else 1)
    out, mag = x.copy(), np.abs(x)
    pairs = np.arange(half)
    iu, iv = (first + 2 * pairs, first + 2 * pairs + 1) if layout == "pairs" else (first + pairs, first + half + pairs)
    u, v = x[..., iu], x[..., iv]
    out[..., iu], out[..., iv] = u * c - v * s, v * c + u * s
    mag[..., iu], mag[..., iv] = np.abs(u * c) + np.abs(v * s), np.abs(v * c) + np.abs(u * s)
    return out, mag


def rotate_tolerance(out, mag, kind):
    """Two products and a sum in fp32, each off by half a step, then the type's half step of that."""
    off = 2.0 ** -23 * mag * (1 + 2.0 ** -20)
    return off + HALF[kind] * (np.abs(out) + off)


def queries(x, w, eps, cs, kind):
    """(result, tolerance) of normalised and turned queries x [T, H, 512].

    The mean of squares: 16 products into one sum per lane and 5 more sums, each off by half a step of at most the
    whole, so 21 * 2^-24, and the rounding of it with eps; the root halves that and is rounded, and two products
    follow: 11 + 4 half steps, taken as 2^-20."""
    n = x / np.sqrt((x * x).mean(-1, keepdims=True) + eps)
    if w is not None:
        n = n * w
    out, mag = rotate(n, cs, NOPE, "pairs", False)
    off = mag * (2.0 ** -20 + 2.0 ** -23)
    return out, off + HALF[kind] * (np.abs(out) + off)


def seen(p, window, first, most):
    """Entries that the token at position p sees, of a table row that holds `most`."""
    begin = max(0, p + 1 - window)
    return list(range(min(first, begin, most))) + list(range(begin, min(p + 1, most)))
