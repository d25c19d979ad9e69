"""Plain 64-bit statements of the training-step operators, for their tests: numpy and integer
arithmetic only, nothing of the library."""
import math

import numpy as np

BLOCK = 256
ACTS = {"none": 0, "relu": 1, "gelu": 2, "silu": 3}
# the largest |act'| over all z, and |act(z)| <= |z|
SLOPE = {"none": 1.0, "relu": 1.0, "gelu": 1.13, "silu": 1.1}
# (rows, in, out) whose backward has several of dw's tiles on each unit that dx's last round leaves idle
SHARED_ROUNDS = [(300, 2304, 768), (256, 4096, 1000), (600, 1024, 2048), (512, 2048, 2048), (300, 4096, 2312)]


def act(z, name):
    if name == "relu":
        return np.maximum(z, 0.0)
    if name == "gelu":
        return 0.5 * z * (1.0 + np.tanh(math.sqrt(2.0 / math.pi) * (z + 0.044715 * z ** 3)))
    if name == "silu":
        return z / (1.0 + np.exp(-z))
    return z


def slope(z, name):
    if name == "relu":
        return (z > 0).astype(np.float64)
    if name == "gelu":
        c = math.sqrt(2.0 / math.pi)
        t = np.tanh(c * (z + 0.044715 * z ** 3))
        return 0.5 * (1.0 + t) + 0.5 * z * (1.0 - t * t) * c * (1.0 + 3 * 0.044715 * z * z)
    if name == "silu":
        s = 1.0 / (1.0 + np.exp(-z))
        return s * (1.0 + z * (1.0 - s))
    return np.ones_like(z)


def round_bf16(x):
    """Round-to-nearest-even bf16 values of fp32 numbers (finite or not), as fp32."""
    b = np.asarray(x, np.float32).view(np.uint32).astype(np.uint64)
    r = ((b + 0x7FFF + ((b >> 16) & 1)) & 0xFFFF0000).astype(np.uint32).view(np.float32)
    return np.where(np.isnan(x), np.float32("nan"), r)


def pcg(x):
    x = (np.asarray(x, np.uint64) * np.uint64(747796405) + np.uint64(2891336453)) & np.uint64(0xFFFFFFFF)
    x = (((x >> ((x >> np.uint64(28)) + np.uint64(4))) ^ x) * np.uint64(277803737)) & np.uint64(0xFFFFFFFF)
    return (x >> np.uint64(22)) ^ x


def random_bits(seed, index, n):
    key = pcg((pcg(np.uint64(seed)) + np.uint64(index)) & np.uint64(0xFFFFFFFF))
    return pcg((np.arange(n, dtype=np.uint64) + key) & np.uint64(0xFFFFFFFF))


def _exponent(top):
    """e of a block whose largest magnitude is `top`: that of top rounded up to 4 significant bits."""
    if top == 0.0:
        return -126
    f, e = math.frexp(top)           # top = f 2^e, f in [1/2, 1)
    e -= 1
    if f * 16 > 15:                  # more than 1.875 2^e
        e += 1
    return min(max(e, -126), 126)


def encode(x, r16, exponent_bits):
    """(codes, scales) of binary32 moments, one value at a time in exact arithmetic: the
    magnitude in steps of the code's last place, in units of 2^-20 of it, plus 16 r + 8."""
    top_field = 2 ** exponent_bits - 1
    n = len(x)
    codes = np.zeros(n, np.uint8)
    scales = np.zeros(-(-n // BLOCK), np.float32)
    for b in range(len(scales)):
        lo, hi = b * BLOCK, min(n, (b + 1) * BLOCK)
        a = np.abs(x[lo:hi].astype(np.float64))
        if not np.isfinite(a).all():
            scales[b] = np.nan
            continue
        e = _exponent(float(a.max()))
        scales[b] = 2.0 ** e
        a = np.ldexp(a, -e)                      # exact: below 2 (below 4 at the end of the range)
        f, k = np.frexp(a)                       # a = f 2^k
        field = np.maximum(k - 1 + top_field, 0)     # exponent field; 0: gradual underflow
        field = np.where(a == 0.0, 0, field)
        unit = np.ldexp(1.0, np.maximum(field, 1) - top_field - 3)  # of the last place
        t = a / unit                             # in last places: 8..16, or below 8 at field 0
        t = np.rint(t * 2.0 ** 20)               # (binary32 keeps 20 bits below the last place)
        q = np.floor((t + 16.0 * r16[lo:hi].astype(np.float64) + 8.0) / 2.0 ** 20)
        c = np.where(field > 0, (field - 1) * 8 + q, q)
        c = np.minimum(c, 2 ** (exponent_bits + 3) - 1).astype(np.uint8)
        if exponent_bits == 4:
            c |= np.where(np.signbit(x[lo:hi]), 0x80, 0).astype(np.uint8)
        codes[lo:hi] = c
    return codes, scales


def decode(codes, scales, exponent_bits):
    top_field = 2 ** exponent_bits - 1
    c = codes.astype(np.int64)
    sign = np.ones(len(c))
    if exponent_bits == 4:
        sign, c = np.where(c >= 128, -1.0, 1.0), c & 127
    field, f = c >> 3, c & 7
    a = np.where(field > 0, np.ldexp(1.0 + f / 8.0, field - top_field), np.ldexp(f / 8.0, 1 - top_field))
    with np.errstate(under="ignore"):
        return (sign * a * np.repeat(scales.astype(np.float64), BLOCK)[:len(c)]).astype(np.float32)


def moments(g, m, v, b1, b2):
    """The new binary32 moments, one rounding per operation."""
    f = np.float32
    with np.errstate(over="ignore", invalid="ignore", under="ignore"):
        m = (m * f(b1)) + (f(1.0 - b1) * g)
        v = (v * f(b2)) + ((f(1.0 - b2) * g) * g)
    return m.astype(f), v.astype(f)


def update(w, m, v, lr, wd, b1, b2, eps, t):
    """The new master weights in 64 bits."""
    w, m, v = (np.asarray(x, np.float64) for x in (w, m, v))
    with np.errstate(over="ignore", invalid="ignore", divide="ignore"):
        return w * (1.0 - lr * wd) - lr * (m / (1.0 - b1 ** t)) / (np.sqrt(v / (1.0 - b2 ** t)) + eps)
