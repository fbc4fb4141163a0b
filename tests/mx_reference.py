"""The microscaled 4-bit operators in NumPy float64, from their definitions (the
oracle of tests/test_mx_*.py; no code of the library).

Layout of an operand: KP = K rounded up to 128; codes rows x KP/2 bytes, even k
in the low half; scales rows x KP/32 bytes."""
import numpy as np

E2M1 = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])
F32, BF16, F16 = 0, 1, 2
TYPES = {"f32": F32, "bf16": BF16, "f16": F16}
# half a step of each type, relative to the value
HALF_STEP = {F32: 2.0 ** -24, BF16: 2.0 ** -8, F16: 2.0 ** -11}   # finfo(type).eps / 2


def padded(K):
    return -(-K // 128) * 128


def to_type(x, kind):
    """float64/float32 -> the nearest value of a type, as float32."""
    x = np.asarray(x, np.float32)
    if kind == F32:
        return x
    if kind == F16:
        with np.errstate(over="ignore"):
            return x.astype(np.float16).astype(np.float32)
    return from_bits(bf16_bits(x))


def bf16_bits(x):
    b = np.ascontiguousarray(x, np.float32).view(np.uint32)
    r = ((b + np.uint32(0x7fff) + ((b >> np.uint32(16)) & np.uint32(1))) >> np.uint32(16)).astype(np.uint16)
    nan = (b & np.uint32(0x7fffffff)) > np.uint32(0x7f800000)
    return np.where(nan, np.uint16(0x7fc0), r)


def from_bits(h):
    return (h.astype(np.uint32) << np.uint32(16)).view(np.float32)


def quantize(x):
    """rows x K (exact values of any type) -> (codes, scales), NumPy uint8."""
    x = np.asarray(x, np.float64)
    rows, K = x.shape
    KP = padded(K)
    z = np.zeros((rows, KP))
    z[:, :K] = x
    neg = np.zeros((rows, KP), bool)
    neg[:, :K] = np.signbit(x)
    z = z.reshape(rows, KP // 32, 32)
    top = np.abs(z).max(axis=2)
    lost = ~np.isfinite(top)
    safe = np.where(lost | (top == 0), 1.0, top)
    exponent = np.frexp(safe)[1] - 1 - 2
    exponent = np.where(top == 0, -127, np.maximum(exponent, -127))
    scales = np.where(lost, 255, exponent + 127).astype(np.uint8)
    with np.errstate(invalid="ignore"):
        m = np.abs(z) * np.ldexp(1.0, -exponent)[:, :, None]
    code = np.zeros(m.shape, np.uint8)
    for n in range(1, 8):   # count the borders below; a value on a border goes to the even code
        border = (E2M1[n - 1] + E2M1[n]) / 2
        with np.errstate(invalid="ignore"):
            code += ((m > border) | ((m == border) & (n % 2 == 0))).astype(np.uint8)
    code |= neg.reshape(z.shape).astype(np.uint8) << 3
    code[lost] = 0
    code = code.reshape(rows, KP // 2, 2)
    return (code[:, :, 0] | (code[:, :, 1] << 4)).astype(np.uint8), scales


def decode(codes, scales, K):
    """Operand -> rows x K float64 (NaN under a scale of 255)."""
    rows = codes.shape[0]
    n = np.empty((rows, codes.shape[1] * 2), np.uint8)
    n[:, 0::2], n[:, 1::2] = codes & 15, codes >> 4
    v = E2M1[n & 7] * np.where(n & 8, -1.0, 1.0)
    s = np.where(scales == 255, np.nan, np.ldexp(1.0, scales.astype(np.int32) - 127))
    return (v * np.repeat(s, 32, axis=1))[:, :K]


def product(a, b, alpha=1.0, beta=0.0, c=None):
    """alpha a b^T + beta c and the sum of magnitudes, float64."""
    r, s = alpha * (a @ b.T), abs(alpha) * (np.abs(a) @ np.abs(b).T)
    if beta != 0:
        r, s = r + beta * c, s + np.abs(beta * c)
    return r, s


def route(logits, top_k, renormalize):
    """float64 weights tokens x experts (0: not chosen; a row of NaN for a NaN or +inf)."""
    T, E = logits.shape
    w = np.zeros((T, E))
    for t in range(T):
        l = logits[t].astype(np.float64)
        if np.isnan(l).any() or (l == np.inf).any():
            w[t] = np.nan
            continue
        if not np.isfinite(l).any():
            continue
        p = np.exp(l - l.max())
        p /= p.sum()
        chosen = [e for e in np.argsort(-l, kind="stable")[:top_k] if np.isfinite(l[e])]
        w[t, chosen] = p[chosen] / (p[chosen].sum() if renormalize else 1.0)
    return w


def moe(x, weights, w1, w2, inter, parts_x, parts_h):
    """x T x H, weights T x E, w1 (E * 2 I) x H and w2 (E * H) x I decoded. Returns
    (Y, bound) in float64: what the sums' and the hidden activations' roundings
    can come to, the rounding of Y itself not counted.

    Each FP32 addition is off by at most 2^-23 of the magnitudes summed (matrix
    instructions may cut off instead of rounding): a gate or up value by
    (terms + 8) 2^-23 sum|w x|. silu has a slope of at most 1.1; silu, the
    products and the weight take 16 roundings at most and the softmax weight
    experts of them. Two bfloat16 parts leave 2^-16 of a hidden value (cut off
    after 8 bits, then rounded), three nothing (2^-24)."""
    T, H = x.shape
    E, I = weights.shape[1], inter
    y, bound = np.zeros((T, H)), np.zeros((T, H))
    u = 2.0 ** -23
    mag = np.zeros((T, H))
    for e in range(E):
        who = [t for t in range(T) if weights[t, e] > 0]
        if not who:
            continue
        wg, wu = w1[e * 2 * I:e * 2 * I + I], w1[e * 2 * I + I:(e + 1) * 2 * I]
        g, v = x[who] @ wg.T, x[who] @ wu.T
        eg = (H * parts_x + 8) * u * (np.abs(x[who]) @ np.abs(wg).T)
        ev = (H * parts_x + 8) * u * (np.abs(x[who]) @ np.abs(wu).T)
        s = g / (1 + np.exp(-g))
        a = s * v * weights[who, e][:, None]
        ea = (1.1 * eg * (np.abs(v) + ev) + np.abs(s) * ev) * weights[who, e][:, None] + \
            (16 + E) * u * np.abs(a)
        ea += np.abs(a) * (2.0 ** -16 if parts_h == 2 else 2.0 ** -24)
        d = w2[e * H:(e + 1) * H]
        y[who] += a @ d.T
        bound[who] += ea @ np.abs(d).T
        mag[who] += (np.abs(a) + ea) @ np.abs(d).T
    k = np.count_nonzero(weights, axis=1).max() if T else 0
    bound += (k * I * parts_h + 16) * u * mag
    y[np.isnan(weights).any(axis=1)] = np.nan
    return y, bound
