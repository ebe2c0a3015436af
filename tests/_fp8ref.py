"""64-bit reference forms for the feed-forward operators' tests, written from
the formulas in numpy; nothing here calls the library."""
import numpy as np

E4M3_HALF_STEP = 2.0 ** -4    # a normal E4M3 value is within this, relative, of what was rounded
E4M3_SUB_HALF = 2.0 ** -10    # a subnormal one within this, in units of the scale


def e4m3_table():
    t = np.zeros(256)
    for c in range(256):
        e, m = (c >> 3) & 15, c & 7
        v = (m / 8) * 2.0 ** -6 if e == 0 else (1 + m / 8) * 2.0 ** (e - 7)
        t[c] = np.nan if (c & 0x7F) == 0x7F else (-v if c & 128 else v)
    return t


TABLE = e4m3_table()


def codes_to_values(q):
    """uint8 codes -> float64."""
    return TABLE[np.asarray(q, dtype=np.uint8)]


def unpack_rows(words, rows, cols):
    """Packed scale words [ceil(cols/512), align(rows, 4)] -> scales [rows, cols/128]."""
    b = np.ascontiguousarray(words).view(np.uint8).reshape(words.shape[0], words.shape[1], 4)
    return 2.0 ** (b.transpose(1, 0, 2).reshape(words.shape[1], -1)[:rows, :cols // 128].astype(np.float64) - 127)


def row_values(q, words):
    """Codes with 1x128 row-group scales -> float64."""
    rows, cols = q.shape
    return codes_to_values(q) * np.repeat(unpack_rows(words, rows, cols), 128, axis=1)


def col_scales(words, rows, cols):
    """Column scales (one per 128 rows of each column) repeated to [rows, cols]."""
    return np.repeat(unpack_rows(words, cols, rows).T, 128, axis=0)


def unused_bytes(words, rows, blocks):
    """The bytes of the packed words that belong to no row or block (must be 0)."""
    b = np.ascontiguousarray(words).view(np.uint8).reshape(words.shape[0], words.shape[1], 4)
    b = b.transpose(1, 0, 2).reshape(words.shape[1], -1)
    return np.concatenate([b[rows:].ravel(), b[:rows, blocks:].ravel()])


def act(g, name):
    if name == "silu":
        return g / (1 + np.exp(-g))
    return 0.5 * g * (1 + np.tanh(np.sqrt(2 / np.pi) * (g + 0.044715 * g ** 3)))


def act_grad(g, name):
    if name == "silu":
        s = 1 / (1 + np.exp(-g))
        return s * (1 + g * (1 - s))
    c = np.sqrt(2 / np.pi)
    t = np.tanh(c * (g + 0.044715 * g ** 3))
    return 0.5 * (1 + t) + 0.5 * g * (1 - t * t) * c * (1 + 3 * 0.044715 * g ** 2)


def check_codes(q, scales, groups_axis, value, slack, what):
    """q: uint8 codes; scales: the scale of every element; value: the exact
    result; slack: how far FP32 arithmetic may be from it, per element.

    Every scale is the rule's for a group maximum within the slack, and every
    code the nearest E4M3 value to a number within the slack of value/scale:
    |code * scale - value| <= half a step + slack."""
    shape = list(value.shape)
    if groups_axis == 1:
        cut = lambda a: a.reshape(shape[0], shape[1] // 128, 128).max(2)  # noqa: E731
        s = scales[:, ::128]
    else:
        cut = lambda a: a.reshape(shape[0] // 128, 128, shape[1]).max(1)  # noqa: E731
        s = scales[::128]
    hi, lo = cut(np.abs(value) + slack), np.maximum(cut(np.abs(value) - slack), 0)
    zero = hi == 0
    assert (s[zero] == 1).all(), "%s: an all-zero group's scale is not 1" % what
    tiny = s == 2.0 ** -127
    assert (zero | (448 * s >= lo)).all(), "%s: scale too small" % what
    assert (zero | tiny | (224 * s < hi)).all(), "%s: scale too large" % what
    got = codes_to_values(q) * scales
    v = np.abs(value) / scales
    step = np.exp2(np.floor(np.log2(np.maximum(v, 2.0 ** -6))) - 3)
    off = np.abs(got - value) - (0.5 * step * scales + slack)
    assert np.isfinite(got).all() and (off <= 1e-12 * np.abs(value)).all(), \
        "%s: a code is %.3g past half a step" % (what, off.max())
