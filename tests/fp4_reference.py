"""Microscaled 4-bit floats and block norms by their definitions, in 64 bits on
the CPU (f32 where the definition names an f32 rounding: numpy's division and
product are correctly rounded)."""
import numpy as np
import torch

BLOCK = {"mx": 32, "nv": 16}
WORD = {"mx": 128, "nv": 64}
VALUES = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])


def gen(seed):
    return torch.Generator(device="cpu").manual_seed(seed)


def randn(g, *shape, std=1.0, mean=0.0, dtype=torch.bfloat16):
    return (torch.randn(*shape, generator=g) * std + mean).to(dtype)


def e2m1(q):
    """Codes of f64 quotients: nearest value, ties to the even code, the sign kept."""
    a = np.minimum(np.abs(q), 6.0)
    upper = np.clip(np.searchsorted(VALUES, a, side="left"), 1, 7)  # VALUES[upper - 1] <= a <= VALUES[upper]
    lo, hi = VALUES[upper - 1], VALUES[upper]
    mid = (lo + hi) / 2
    code = np.where((a > mid) | ((a == mid) & (upper % 2 == 0)), upper, upper - 1)
    return (code | np.where(np.signbit(q), 8, 0)).astype(np.uint8)


def e4m3(s):
    """Bytes of f64 numbers >= 0: nearest, ties to even, at most 448."""
    s = np.asarray(s, dtype=np.float64)
    step = np.ldexp(1.0, np.maximum(np.frexp(s)[1] - 4, -9))
    v = np.minimum(np.rint(s / step) * step, 448.0)
    _, e = np.frexp(v)
    normal = v >= 2.0 ** -6
    return np.where(normal, ((e + 6) << 3) | (np.rint(np.ldexp(v, 4 - e)).astype(np.int64) - 8),
                    np.rint(v * 512).astype(np.int64)).astype(np.uint8)


def e4m3_value(b):
    b = b.astype(np.int64)
    v = np.where(b >= 8, np.ldexp((b % 8 + 8).astype(np.float64), b // 8 - 10), np.ldexp((b % 8).astype(np.float64), -9))
    return np.where(b == 0x7f, np.nan, v)


def block_scales(x, fmt, t):
    """(bytes, divisors in f32) of the blocks of x, f32 [M, K]."""
    b = np.abs(x.reshape(x.shape[0], -1, BLOCK[fmt]))
    bad = ~np.isfinite(b).all(-1)
    amax = np.where(bad, np.float32(0), b.max(-1)).astype(np.float32)
    if fmt == "mx":
        e = np.maximum(np.where(amax > 0, np.frexp(amax.astype(np.float64))[1] - 1, -200) - 2, -127)
        return np.where(bad, 255, e + 127).astype(np.uint8), np.ldexp(1.0, e)
    byte = e4m3(np.float32(amax) / (np.float32(6) * np.float32(t)))
    d = e4m3_value(byte).astype(np.float32) * np.float32(t)
    return np.where(bad, 0x7f, byte).astype(np.uint8), d.astype(np.float64)


def quantize(x, fmt, t=1.0):
    """x f32 [M, K] -> (codes [M, K], scales by row).  Codes of blocks with a NaN scale are of no consequence."""
    x = np.asarray(x, dtype=np.float32)
    scales, d = block_scales(x, fmt, t)
    bad = scales == (255 if fmt == "mx" else 0x7f)
    b = x.reshape(x.shape[0], -1, BLOCK[fmt])
    with np.errstate(all="ignore"):
        q = np.where((d > 0)[..., None], (b / d[..., None].astype(np.float32)).astype(np.float64), np.copysign(0.0, b))
        q = np.where(bad[..., None], 0.0, q)
    return e2m1(q).reshape(x.shape), scales


def pack(codes):
    return (codes[:, 0::2] | codes[:, 1::2] << 4).astype(np.uint8)


def unpack(packed):
    return np.stack([packed & 15, packed >> 4], -1).reshape(packed.shape[0], -1)


def values(codes, scales, fmt):
    """Code * block scale, f64 [M, K] (without a tensor's scale)."""
    v = VALUES[codes & 7] * np.where(codes & 8, -1.0, 1.0)
    s = np.where(scales == 255, np.nan, np.ldexp(1.0, scales.astype(np.int64) - 127)) if fmt == "mx" else e4m3_value(scales)
    return v * np.repeat(s, BLOCK[fmt], axis=1)


def tile(scales, fmt):
    """Scales by row -> tiled (rows past the last: 0)."""
    rows, blocks = scales.shape
    words = -(-blocks // 4)
    tiles = -(-rows // 128)
    full = np.zeros((tiles * 128, words * 4), np.uint8)
    full[:rows, :blocks] = scales
    # [tile, quarter, row, word, 4] -> [tile, word, row, quarter, 4]
    return full.reshape(tiles, 4, 32, words, 4).transpose(0, 3, 2, 1, 4).reshape(-1)


def untile(tiled, rows, K, fmt):
    words = -(-K // WORD[fmt])
    tiles = -(-rows // 128)
    full = np.asarray(tiled).reshape(tiles, words, 32, 4, 4).transpose(0, 3, 2, 1, 4).reshape(tiles * 128, words * 4)
    assert (full[:rows, K // BLOCK[fmt]:] == 0).all(), "scales past K"
    return full[:rows, :K // BLOCK[fmt]]


def product(x, w, alpha, bias=None, residual=None):
    """(y, bound): f64 product of values x [M, K], w [N, K], and how far a kernel's bf16 result may be from it.

    Half a bf16 step, 2^-8 of the result.  In f32 before it: a product of two codes and scales has at most 16
    bits and is exact; each addition of the sum is off by at most 2^-23 (a truncating adder) of what is added so
    far, at most S = sum |x w|: of a chain of at most K / 16 + 32 additions (blocks of an instruction, instructions,
    parts); then alpha (itself rounded: twice 2^-24), bias and residual at 2^-24 each of the sum of magnitudes."""
    y = alpha * (x @ w.T)
    S = abs(alpha) * (np.abs(x) @ np.abs(w).T)
    parts = S.copy()
    for extra in (bias, residual):
        if extra is not None:
            y = y + extra
            parts = parts + np.abs(extra)
    f32 = (x.shape[1] / 16 + 32) * 2.0 ** -23 * S + 5 * 2.0 ** -24 * parts
    return y, 2.0 ** -8 * (np.abs(y) + f32) + f32


def assert_product(got, want, bound, what="y"):
    got = got.double().cpu().numpy() if torch.is_tensor(got) else got
    nan = np.isnan(want)
    assert np.array_equal(np.isnan(got), nan), f"{what}: NaN in other places"
    far = np.where(nan, 0.0, np.abs(np.where(nan, 0.0, got) - np.where(nan, 0.0, want)) - np.where(nan, 0.0, bound))
    worst = np.unravel_index(np.argmax(far), far.shape)
    assert far[worst] <= 0, f"{what}{worst}: {got[worst]} instead of {want[worst]}, bound {bound[worst]}"


def block_norm(x, branch=None, post_weight=None, gate=None, x_factor=1.0, branch_factor=1.0, norm="rms", weight=None,
               bias=None, scale=None, shift=None, tokens_per_group=0, eps=1e-6):
    """(h, n) in f64, tensors in and out."""
    def f64(t):
        return None if t is None else t.double().cpu()
    x, branch, post_weight, gate, weight, bias, scale, shift = map(f64, (x, branch, post_weight, gate, weight, bias, scale, shift))
    T = x.shape[0]
    rows = torch.arange(T) // tokens_per_group if tokens_per_group > 0 else torch.zeros(T, dtype=torch.long)
    h = x_factor * x
    if branch is not None:
        b = branch
        if post_weight is not None:
            b = b / (b.square().mean(-1, keepdim=True) + eps).sqrt() * post_weight
        if gate is not None:
            b = b * gate[rows]
        h = h + branch_factor * b
    n = h - h.mean(-1, keepdim=True) if norm == "layer" else h
    n = n / (n.square().mean(-1, keepdim=True) + eps).sqrt()
    if weight is not None:
        n = n * weight
    if bias is not None:
        n = n + bias
    if scale is not None:
        n = n * (1 + scale[rows])
    if shift is not None:
        n = n + shift[rows]
    return h, n


def norm_bounds(h, n, a):
    """How far f32 arithmetic may be from (h, n) of block_norm(**a), before its last rounding.

    u = 2^-24, the row's width H.  h: five roundings of its two terms, and the branch's own norm (a sum of H squares in
    any order, at most H / 8 + 24 deep here: that many u, halved by the root; the root and products 4 u).  n: h's
    errors, the mean's ((H / 8 + 24) u of the mean magnitude), the variance's likewise, and five u of each term."""
    u = 2.0 ** -24
    x, branch = a["x"].double().cpu(), a.get("branch")
    H = x.shape[1]
    depth = (H / 8 + 24) * u
    xf, bf = abs(a.get("x_factor", 1.0)), a.get("branch_factor", 1.0)
    terms = xf * x.abs()
    err = 5 * u * terms
    if branch is not None:
        part = (h - a.get("x_factor", 1.0) * x).abs()
        terms = terms + part
        err = err + (8 * u + (depth if a.get("post_weight") is not None else 0.0)) * part + u * terms
    std = (h - h.mean(-1, keepdim=True)).square().mean(-1, keepdim=True) if a.get("norm") == "layer" else h.square().mean(-1, keepdim=True)
    inv = 1 / (std + a.get("eps", 1e-6)).sqrt()
    rows = torch.arange(x.shape[0]) // a["tokens_per_group"] if a.get("tokens_per_group", 0) > 0 else torch.zeros(x.shape[0], dtype=torch.long)
    factor = torch.ones_like(h)
    if a.get("weight") is not None:
        factor = factor * a["weight"].double().cpu().abs()
    if a.get("scale") is not None:
        factor = factor * (1 + a["scale"].double().cpu()[rows]).abs()
    c = h
    e = err
    if a.get("norm") == "layer":
        c = h - h.mean(-1, keepdim=True)
        e = e + err.mean(-1, keepdim=True) + depth * h.abs().mean(-1, keepdim=True) + u * h.abs()
    # of the row's statistic, relative
    stat = ((c.abs() * e).mean(-1, keepdim=True) * inv * inv) + depth
    y = c.abs() * inv * factor
    en = e * inv * factor + (stat + 6 * u) * y + 4 * u * (y + n.abs())
    for extra, f in (("bias", a.get("scale")), ("shift", None)):
        if a.get(extra) is not None:
            v = a[extra].double().cpu().abs()
            v = v[rows] if extra == "shift" else v
            if f is not None:
                v = v * (1 + f.double().cpu()[rows]).abs()
            en = en + 4 * u * v
    return err, en


def assert_codes_of(codes, scales, lo, hi, fmt, t, what="codes"):
    """Codes and scales (by row) are those of some f32 values between lo and hi (f64 [M, K]): each block's scale is one
    between those of the smallest and the largest amax, each code between those of lo and hi at that scale."""
    M, K = lo.shape
    mag_lo = np.where((lo < 0) & (hi > 0), 0.0, np.minimum(np.abs(lo), np.abs(hi)))
    mag_hi = np.maximum(np.abs(lo), np.abs(hi))
    f32lo, f32hi = mag_lo.astype(np.float32), mag_hi.astype(np.float32)
    s_lo, _ = block_scales(np.nextafter(f32lo, np.float32(0)), fmt, t)
    s_hi, _ = block_scales(np.nextafter(f32hi, np.float32(np.inf)), fmt, t)
    assert ((s_lo <= scales) & (scales <= s_hi)).all(), f"{what}: a scale"
    d = np.ldexp(1.0, scales.astype(np.int64) - 127) if fmt == "mx" else e4m3_value(scales) * np.float64(np.float32(t))
    d = np.repeat(d, BLOCK[fmt], axis=1)
    v = VALUES[codes & 7] * np.where(codes & 8, -1.0, 1.0)
    with np.errstate(all="ignore"):
        eps = 2.0 ** -22  # of the quotient's and the divisor's roundings
        q_lo, q_hi = np.where(d > 0, lo / d, 0.0), np.where(d > 0, hi / d, 0.0)
    def value(q):
        c = e2m1(q)
        return VALUES[c & 7] * np.where(c & 8, -1.0, 1.0)
    low, high = value(q_lo - eps * np.abs(q_lo)), value(q_hi + eps * np.abs(q_hi))
    bad = (v < low) | (v > high)
    assert not bad.any(), f"{what}: {int(bad.sum())} codes, first at {tuple(np.argwhere(bad)[0])}"
