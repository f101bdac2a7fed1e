"""The attention operators from their definitions in 64 bits (plain torch on any
device), the inputs of their tests and the bounds their outputs must keep."""
import math

import torch

F64 = torch.float64
U = 2.0 ** -8  # bf16 unit roundoff: 8 significant bits, half a spacing of 2^-7 in [1, 2)


def gen(seed):
    g = torch.Generator(device="cpu")
    g.manual_seed(seed)
    return g


def randn(g, *shape, std=1.0, dtype=torch.bfloat16):
    return (torch.randn(*shape, generator=g) * std).to(dtype)


def rope_table(max_pos, rot):
    inv = 10000.0 ** (-torch.arange(0, rot, 2, dtype=F64) / rot)
    ang = torch.arange(max_pos, dtype=F64)[:, None] * inv[None]
    return torch.cat([ang.cos(), ang.sin()], 1).float()


def norm_rope(x, w, eps, table, pos, mode):
    """x [T, H, D] -> f64; w, table may be None."""
    y = x.to(F64)
    if w is not None:
        y = y / torch.sqrt((y ** 2).mean(-1, keepdim=True) + eps) * w.to(F64)
    if table is None:
        return y
    r = table.shape[1]
    c = table.to(F64)[pos.long(), :r // 2]
    s = table.to(F64)[pos.long(), r // 2:]
    out = y.clone()
    for i in range(r // 2):
        a, b = (i, i + r // 2) if mode == "half" else (2 * i, 2 * i + 1)
        out[:, :, a] = y[:, :, a] * c[:, i, None] - y[:, :, b] * s[:, i, None]
        out[:, :, b] = y[:, :, b] * c[:, i, None] + y[:, :, a] * s[:, i, None]
    return out


def assert_norm_rope(got, ref, what=""):
    """One rounding to bf16 (U of the value) after f32 arithmetic: the norm's factor, weight and rotation are
    at most 16 roundings (and rsqrt's 2 ulp) of numbers no larger than twice the row's largest."""
    got, ref = got.to(F64).cpu(), ref.cpu()
    top = ref.abs().amax(-1, keepdim=True)
    bound = U * ref.abs() + 2 * 20 * 2.0 ** -24 * top + 1e-30
    bad = (got - ref).abs() > bound * (1 + 1e-6)
    assert torch.isfinite(got).all() and not bad.any(), \
        f"{what}: {int(bad.sum())} of {bad.numel()} off, worst {((got - ref).abs() / bound).max():.2f} of the bound"


def softmax_av(q, k, v, last, scale):
    """Rows q [R, D] over keys k, v [n, D]; row r sees keys 0 .. last[r] - 1 -> (out, out with |v|), f64."""
    q, k, v = q.to(F64), k.to(F64), v.to(F64)
    R, n = q.shape[0], k.shape[0]
    if n == 0:
        z = torch.zeros(R, q.shape[1], dtype=F64, device=q.device)
        return z, z.clone()
    x = scale * (q @ k.T)
    seen = torch.arange(n, device=q.device)[None] < last[:, None]
    x = torch.where(seen, x, torch.full_like(x, -math.inf))
    m = x.amax(1, keepdim=True)
    p = torch.exp(x - torch.where(torch.isfinite(m), m, torch.zeros_like(m)))
    s = p.sum(1, keepdim=True)
    p = p / torch.where(s > 0, s, torch.ones_like(s))
    return p @ v, p @ v.abs()


def attend(q, keys, values, last, scale):
    """q [B, Lq, Hq, D]; keys, values: per sequence [n, Hkv, D]; last [B][Lq] -> (out, out of |v|) f64."""
    B, Lq, Hq, D = q.shape
    out = torch.zeros(q.shape, dtype=F64, device=q.device)
    mag = out.clone()
    for b in range(B):
        H = keys[b].shape[1]
        G = Hq // H
        rows = torch.as_tensor(last[b], device=q.device).repeat_interleave(G)
        for h in range(H):
            o, m = softmax_av(q[b, :, h * G:(h + 1) * G].reshape(Lq * G, D), keys[b][:, h], values[b][:, h],
                              rows, scale)
            out[b, :, h * G:(h + 1) * G] = o.view(Lq, G, D)
            mag[b, :, h * G:(h + 1) * G] = m.view(Lq, G, D)
    return out, mag


def assert_attention(got, ref, mag, what=""):
    """out = sum p v / sum p.  The probabilities enter the second product as bf16, each off by U at most: U of
    sum p |v| / sum p.  Storing the output adds U of it.  The rest is f32: scores of a few units off by some
    2^-20, the exponential and the sums by a few 2^-22 each: below 2^-14 of the same sum."""
    got = got.to(F64)
    bound = U * (1 + U) * (mag + ref.abs()) + 2.0 ** -14 * mag + 1e-30
    bad = ~((got - ref).abs() <= bound)
    assert not bad.any(), (f"{what}: {int(bad.sum())} of {bad.numel()} off, "
                           f"worst {((got - ref).abs() / bound).nan_to_num(1e9).max():.2f} of the bound")


class Paged:
    """A paged cache with a shared prefix and each sequence's own tokens, on pages in any order; every row that
    no sequence uses holds `junk`."""

    def __init__(self, seed, B, H, D, page, prefix, lens, junk=float("nan"), max_len=None, std=1.0, spare=2):
        g = gen(seed)
        self.prefix_len, self.lens, self.page = prefix, lens, page
        self.max_len = max(lens) if max_len is None else max_len
        npre = -(-prefix // page)
        per = [-(-n // page) for n in lens]
        pages = npre + sum(per) + spare
        order = torch.randperm(pages, generator=g)
        self.k_cache = torch.full((pages, H, page, D), junk, dtype=torch.bfloat16)
        self.v_cache = self.k_cache.clone()
        width = max(1, -(-self.max_len // page))
        self.block_table = torch.full((B, width), -7, dtype=torch.int32)  # entries past a length are not read
        self.prefix_pages = order[:npre].to(torch.int32)
        self.pk, self.pv = randn(g, prefix, H, D, std=std), randn(g, prefix, H, D)
        self._fill(self.prefix_pages.tolist(), self.pk, self.pv)
        self.k, self.v, at = [], [], npre
        for b in range(B):
            mine = order[at:at + per[b]].to(torch.int32)
            at += per[b]
            self.block_table[b, :per[b]] = mine
            k, v = randn(g, lens[b], H, D, std=std), randn(g, lens[b], H, D)
            self._fill(mine.tolist(), k, v)
            self.k.append(k)
            self.v.append(v)
        self.seq_lens = torch.tensor(lens, dtype=torch.int32)

    def _fill(self, pages, k, v):
        for i, p in enumerate(pages):
            n = min(self.page, k.shape[0] - i * self.page)
            self.k_cache[p, :, :n] = k[i * self.page:i * self.page + n].transpose(0, 1)
            self.v_cache[p, :, :n] = v[i * self.page:i * self.page + n].transpose(0, 1)

    def reference(self, q, scale):
        """(out, out of |v|) in 64 bits on q's device."""
        Lq = q.shape[1]
        dev = q.device
        keys = [torch.cat([self.pk, k]).to(dev) for k in self.k]
        values = [torch.cat([self.pv, v]).to(dev) for v in self.v]
        last = [[self.prefix_len + max(0, n - Lq + i + 1) for i in range(Lq)] for n in self.lens]
        return attend(q, keys, values, last, scale)

    def to(self, dev):
        for name in ("k_cache", "v_cache", "block_table", "prefix_pages", "seq_lens"):
            setattr(self, name, getattr(self, name).to(dev))
        return self
