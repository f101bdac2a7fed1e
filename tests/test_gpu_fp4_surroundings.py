"""Random sizes with every output and workspace in the middle of marked memory: the values against the definitions in
64 bits, and the memory around them as it was."""
import random

import numpy as np
import pytest
import torch

import fp4_reference as ref
import swiglu_mlp_group_gb300 as ck
from gpu_helpers import device, poll_ok

pytestmark = pytest.mark.gpu

MARK, AROUND = 0xa5, 4096


class Marked:
    """Tensors inside marked memory."""

    def __init__(self, dev):
        self.dev, self.made = dev, []

    def __call__(self, shape, dtype):
        n = int(np.prod(shape)) * dtype.itemsize
        raw = torch.full((n + 2 * AROUND,), MARK, dtype=torch.uint8, device=self.dev)
        self.made.append((raw, n))
        return raw[AROUND:AROUND + n].view(dtype).view(shape)

    def check(self):
        torch.cuda.synchronize()
        for raw, n in self.made:
            assert (raw[:AROUND] == MARK).all() and (raw[AROUND + n:] == MARK).all(), "written outside an output"


def log_int(rng, lo, hi, of=1):
    return max(lo, min(hi, round(lo * (hi / lo) ** rng.random()))) // of * of


def weight(g, rows, K, fmt, t, dev):
    w = ref.randn(g, rows, K, std=K ** -0.5)
    return ck.fp4_quantize(w.to(dev), fmt, scale=t), ref.values(*ref.quantize(w.float().numpy(), fmt, t), fmt)


@pytest.mark.parametrize("seed", range(24))
def test_linear(seed):
    dev = device()
    rng, g = random.Random(seed), ref.gen(seed)
    fmt = rng.choice(["mx", "nv"])
    t = 1.0 if fmt == "mx" else 0.004
    M, K, N = log_int(rng, 1, 700), log_int(rng, 32, 6000, 32), log_int(rng, 8, 900, 8)
    near = Marked(dev)
    (w, ws), wv = weight(g, N, K, fmt, t, dev)
    x = ref.randn(g, M, K)
    codes, scales = near((M, K // 2), torch.uint8), near((int(ck.lib().ck_fp4_scale_bytes(ck._FP4S[fmt], M, K)),), torch.uint8)
    ck.fp4_quantize(x.to(dev), fmt, scale=t, codes=codes, scales=scales)
    rc, rs = ref.quantize(x.float().numpy(), fmt, t)
    assert np.array_equal(ref.unpack(codes.cpu().numpy()), rc) and np.array_equal(ref.untile(scales.cpu().numpy(), M, K, fmt), rs)
    alpha = float(np.float32(t) * np.float32(t))
    bias = ref.randn(g, N) if rng.random() < 0.5 else None
    residual = ref.randn(g, M, N) if rng.random() < 0.5 else None
    want, bound = ref.product(ref.values(rc, rs, fmt), wv, alpha, *(None if v is None else v.double().numpy() for v in (bias, residual)))
    on = lambda v: None if v is None else v.to(dev)  # noqa: E731
    y = near((M, N), torch.bfloat16)
    ck.fp4_gemm(codes, scales, w, ws, fmt, alpha=alpha, bias=on(bias), residual=on(residual), out=y)
    ref.assert_product(y, want, bound, f"product {M} x {K} -> {N}")
    z, work = near((M, N), torch.bfloat16), near((int(ck.lib().ck_fp4_linear_workspace_bytes(M, K, ck._FP4S[fmt])),), torch.uint8)
    if residual is not None:
        z.copy_(residual)
    ck.fp4_linear(x.to(dev), w, ws, fmt, x_scale=t, w_scale=t, bias=on(bias), residual=None if residual is None else z, out=z,
                  workspace=work)
    ref.assert_product(z, want, bound, f"linear {M} x {K} -> {N}")
    poll_ok()
    near.check()


@pytest.mark.parametrize("seed", range(16))
def test_mlp(seed):
    """Against the library's own two linears, which the test above holds to the definition."""
    dev = device()
    rng, g = random.Random(100 + seed), ref.gen(100 + seed)
    fmt = rng.choice(["mx", "nv"])
    t = 1.0 if fmt == "mx" else 0.004
    M, H, I = log_int(rng, 1, 700), log_int(rng, 32, 1200, 32), log_int(rng, 32, 1500, rng.choice([32, 64]))
    I = max(I, 32)
    near = Marked(dev)
    (gu, gus), _ = weight(g, 2 * I, H, fmt, t, dev)
    (d, ds), _ = weight(g, H, I, fmt, t, dev)
    x = ref.randn(g, M, H).to(dev)
    y = near((M, H), torch.bfloat16)
    work = near((int(ck.lib().ck_fp4_swiglu_mlp_workspace_bytes(M, H, I, ck._FP4S[fmt])),), torch.uint8)
    ck.fp4_swiglu_mlp(x, gu, gus, d, ds, fmt, t, t, t, t, residual=x, out=y, workspace=work)
    h = ck.fp4_linear(x, gu, gus, fmt, x_scale=t, w_scale=t)
    assert torch.equal(y, ck.fp4_linear(h, d, ds, fmt, x_scale=t, w_scale=t, act="swiglu", residual=x)), (M, H, I)
    poll_ok()
    near.check()


@pytest.mark.parametrize("seed", range(24))
def test_norm(seed):
    dev = device()
    rng, g = random.Random(200 + seed), ref.gen(200 + seed)
    fmt = rng.choice(["mx", "nv"])
    t = 1.0 if fmt == "mx" else 0.004
    T, H = log_int(rng, 1, 900), log_int(rng, 32, 9000, 32)
    per = rng.choice([0, 1, log_int(rng, 1, T)])
    rows = -(-T // per) if per else 1
    mod = ref.randn(g, rows, 3 * H, std=0.3)
    a = dict(x=ref.randn(g, T, H), branch=ref.randn(g, T, H), norm=rng.choice(["rms", "layer"]), tokens_per_group=per,
             weight=ref.randn(g, H, std=0.2, mean=1.0))
    for name, v in (("gate", mod[:, :H]), ("scale", mod[:, H:2 * H]), ("shift", mod[:, 2 * H:]),
                    ("post_weight", ref.randn(g, H, mean=1.0)), ("bias", ref.randn(g, H))):
        if rng.random() < 0.5:
            a[name] = v
    if not any(k in a for k in ("gate", "scale", "shift")):
        a["tokens_per_group"] = 0
    near = Marked(dev)
    d = {k: v.to(dev) if torch.is_tensor(v) else v for k, v in a.items()}
    wide = near((T, 2 * H), torch.bfloat16)
    h, n = wide[:, :H], near((T, H), torch.bfloat16)
    ck.block_norm(**d, h_out=h, n_out=n)
    wh, wn = ref.block_norm(**a)
    eh, en = ref.norm_bounds(wh, wn, a)
    for got, want, e in ((h, wh, eh), (n, wn, en)):
        assert ((got.double().cpu() - want).abs() <= 2.0 ** -8 * (want.abs() + e) + e).all()
    assert (wide[:, H:].contiguous().view(torch.uint8) == MARK).all()
    codes, scales = near((T, H // 2), torch.uint8), near((int(ck.lib().ck_fp4_scale_bytes(ck._FP4S[fmt], T, H)),), torch.uint8)
    ck.block_norm_fp4(**d, fmt=fmt, n_scale=t, codes=codes, scales=scales)
    lo, hi = (wn - en).numpy(), (wn + en).numpy()
    ref.assert_codes_of(ref.unpack(codes.cpu().numpy()), ref.untile(scales.cpu().numpy(), T, H, fmt), lo, hi, fmt, t)
    poll_ok()
    near.check()
