"""Quantization to microscaled 4-bit floats, the product, the linear and the MLP
against their definitions in 64 bits."""
import numpy as np
import pytest
import torch

import fp4_reference as ref
import swiglu_mlp_group_gb300 as ck
from gpu_helpers import device, poll_ok

pytestmark = pytest.mark.gpu

T = {"mx": 1.0, "nv": 0.0037}  # tensor scales
FMTS = ["mx", "nv"]


def quantized(x, fmt, t, act="none"):
    """(codes [M, K], scales by row) of the kernel."""
    codes, scales = ck.fp4_quantize(x, fmt, scale=t, act=act)
    K = 2 * codes.shape[1]
    return ref.unpack(codes.cpu().numpy()), ref.untile(scales.cpu().numpy(), x.shape[0], K, fmt)


def check_quantize(x, fmt, t):
    codes, scales = quantized(x, fmt, t)
    want, want_scales = ref.quantize(x.float().cpu().numpy(), fmt, t)
    assert np.array_equal(scales, want_scales)
    keep = np.repeat(want_scales != (255 if fmt == "mx" else 0x7f), ref.BLOCK[fmt], axis=1)
    assert np.array_equal(codes[keep], want[keep])
    poll_ok()


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("M,K", [(1, 32), (1, 64), (3, 96), (5, 256), (33, 288), (130, 1056), (2, 32768)])
def test_quantize(M, K, fmt, dtype):
    dev = device()
    x = ref.randn(ref.gen(M + K), M, K, dtype=dtype).to(dev)
    x[:, 7::41] *= 20
    for t in ([1.0] if fmt == "mx" else [0.0037, 2.0 ** -8, 1.0, 2.0 ** -60]):
        check_quantize(x, fmt, t)


@pytest.mark.parametrize("fmt", FMTS)
def test_quantize_borders(fmt):
    """Every bf16 mantissa over a range of exponents in blocks of every amax mantissa, on tensor scales that put many
    of them on the borders of codes: 128 blocks x 512 values."""
    dev = device()
    bits = torch.arange(0x3b80, 0x4180, dtype=torch.int32)  # 2^-8 .. 16
    v = bits.to(torch.int16).view(torch.bfloat16)
    b = ref.BLOCK[fmt]
    rows = []
    for top in range(0x4100, 0x4180):  # 8 .. 16: the largest of each block
        m = torch.tensor([top], dtype=torch.int16).view(torch.bfloat16)
        vals = v[v.float() <= m.float()]
        vals = vals[:vals.numel() // (b - 1) * (b - 1)].view(-1, b - 1)
        rows.append(torch.cat([m.expand(vals.shape[0], 1), vals], 1).flatten())
    width = min(r.numel() for r in rows) // 32 * 32
    x = torch.stack([r[:width] for r in rows]).to(dev)
    x[::2] *= -1
    for t in ([1.0] if fmt == "mx" else [1.0, 2.0 ** -9, 45.0 / 2688.0, 0.01]):
        check_quantize(x, fmt, t)


@pytest.mark.parametrize("fmt", FMTS)
def test_quantize_extremes(fmt):
    """Zeros of both signs, numbers from the smallest to the largest, blocks whose scale is cut off at either end."""
    dev = device()
    g = ref.gen(9)
    x = ref.randn(g, 40, 128, dtype=torch.float32)
    e = torch.linspace(-140, 127, 40).round()[:, None]
    x = (x * torch.exp2(e.double())).float().clamp(-3.3e38, 3.3e38)
    x[3] = 0
    x[4, :64] = -0.0
    x[5, 1:64] = 0
    for dtype in (torch.float32, torch.bfloat16):
        y = x.to(dtype).to(dev)
        y = torch.where(torch.isfinite(y), y, torch.full_like(y, 1e38))
        for t in ([1.0] if fmt == "mx" else [1.0, 2.0 ** 60, 2.0 ** -60, 0.0037]):
            check_quantize(y, fmt, t)


@pytest.mark.parametrize("fmt", FMTS)
def test_quantize_not_finite(fmt):
    """A NaN or an infinity marks its own block and no other."""
    dev = device()
    x = ref.randn(ref.gen(3), 6, 192)
    x[0, 5], x[1, 33], x[2, 64], x[3, 191], x[4, 100] = float("nan"), float("inf"), -float("inf"), float("nan"), -float("nan")
    check_quantize(x.to(dev), fmt, T[fmt])
    check_quantize(x.float().to(dev), fmt, T[fmt])


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("M,K", [(1, 32), (37, 416)])
def test_quantize_swiglu(M, K, fmt):
    """silu(gate) * up in f32: a few units in the last place (the exponential and the reciprocal 2^-22 each, the
    rest 2^-24 each: 2^-20 in all), and e^-gate's own argument, off by 2^-24 |gate|."""
    dev = device()
    x = ref.randn(ref.gen(K), M, 2 * K, std=2.0)
    gate, up = x[:, :K].double().numpy(), x[:, K:].double().numpy()
    a = gate / (1 + np.exp(-gate)) * up
    far = np.abs(a) * (2.0 ** -20 + 2.0 ** -23 * np.abs(gate))
    codes, scales = quantized(x.to(dev), fmt, T[fmt], act="swiglu")
    ref.assert_codes_of(codes, scales, a - far, a + far, fmt, T[fmt])
    poll_ok()


@pytest.mark.parametrize("fmt", FMTS)
def test_quantize_rows_apart(fmt):
    """A view of a packed projection's rows, and buffers of the caller's whose rest stays as it was."""
    dev = device()
    wide = ref.randn(ref.gen(1), 70, 640).to(dev)
    x = wide[:, 64:64 + 352]
    codes, scales = ck.fp4_quantize(x, fmt, scale=T[fmt])
    again, scales_again = ck.fp4_quantize(x.contiguous(), fmt, scale=T[fmt])
    K, rows = 352, 70
    assert torch.equal(codes, again)
    assert np.array_equal(ref.untile(scales.cpu().numpy(), rows, K, fmt), ref.untile(scales_again.cpu().numpy(), rows, K, fmt))
    own = torch.full((scales.numel() + 64,), 0xa5, dtype=torch.uint8, device=dev)
    ck.fp4_quantize(x, fmt, scale=T[fmt], scales=own)
    got = own.cpu().numpy()
    assert (got[scales.numel():] == 0xa5).all()
    # words of rows past the last are left as they were
    words = -(-K // ref.WORD[fmt])
    rest = got[:scales.numel()].reshape(1, words, 32, 4, 4).transpose(0, 3, 2, 1, 4).reshape(128, -1)[rows:]
    assert (rest == 0xa5).all()
    poll_ok()


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("rows,K", [(1, 32), (127, 96), (129, 256), (300, 4128)])
def test_tile_scales(rows, K, fmt):
    dev = device()
    s = torch.randint(0, 256, (rows, K // ref.BLOCK[fmt]), generator=ref.gen(K), dtype=torch.uint8)
    tiled = ck.fp4_tile_scales(s.to(dev), fmt)
    assert np.array_equal(ref.untile(tiled.cpu().numpy(), rows, K, fmt), s.numpy())
    poll_ok()


def operand(g, rows, K, fmt, std=1.0):
    """(packed codes, tiled scales, values f64) of random values on the device."""
    x = ref.randn(g, rows, K, std=std, dtype=torch.float32).numpy()
    codes, scales = ref.quantize(x, fmt, T[fmt])
    dev = device()
    tiled = ref.tile(scales, fmt)
    # words of rows past the last hold what they may hold: anything
    full = np.zeros((-(-rows // 128) * 128, scales.shape[1]), np.uint8)
    full[:rows] = 1
    pad = ref.tile(full, fmt) == 0
    words = ref.tile(np.ones_like(full), fmt) == 1
    tiled = np.where(pad & words, 0x7f if fmt == "nv" else 0xff, tiled).astype(np.uint8)
    return torch.from_numpy(ref.pack(codes)).to(dev), torch.from_numpy(tiled).to(dev), ref.values(codes, scales, fmt)


def check_gemm(M, K, N, fmt, bias=False, residual=False, seed=0):
    dev = device()
    g = ref.gen(M * 7 + K * 3 + N + seed)
    xq, xs, xv = operand(g, M, K, fmt)
    wq, ws, wv = operand(g, N, K, fmt, std=K ** -0.5)
    b = ref.randn(g, N) if bias else None
    r = ref.randn(g, M, N) if residual else None
    alpha = T[fmt] * T[fmt]
    y = ck.fp4_gemm(xq, xs, wq, ws, fmt, alpha=alpha, bias=None if b is None else b.to(dev),
                    residual=None if r is None else r.to(dev))
    poll_ok()
    want, bound = ref.product(xv, wv, float(np.float32(alpha)), None if b is None else b.double().numpy(),
                              None if r is None else r.double().numpy())
    ref.assert_product(y, want, bound)
    return y


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("K", [32, 64, 96, 128, 160, 192, 256, 288, 512, 1056, 4096])
def test_gemm_columns(K, fmt):
    check_gemm(5, K, 136, fmt, bias=True)


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("M", [1, 2, 7, 8, 9, 15, 16, 17, 31, 32, 33, 63, 64, 65, 127, 128, 129, 255, 256, 257, 300, 513])
def test_gemm_tokens(M, fmt):
    check_gemm(M, 544, 264, fmt, residual=True)


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("N", [8, 16, 120, 128, 136, 184, 192, 200, 256, 392, 1000, 2056])
@pytest.mark.parametrize("M", [3, 300])
def test_gemm_rows(M, N, fmt):
    check_gemm(M, 320, N, fmt)


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("M,K,N", [(1, 12288, 4096), (8, 4096, 12288), (48, 8192, 1032), (200, 16384, 520), (640, 4128, 2080),
                                   (2049, 1024, 1544)])
def test_gemm_large(M, K, N, fmt):
    check_gemm(M, K, N, fmt, bias=True, residual=True)


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("M,K,N,bias,residual", [(2048, 352, 3400, False, False), (1999, 256, 3256, True, False), (1801, 288, 3400, False, True),
                                                 (2041, 96, 3272, True, True), (4100, 64, 3456, True, True)])
def test_gemm_many_tiles(M, K, N, fmt, bias, residual):
    """Enough tiles that each holds twice the rows of W, whose second half ends inside N, at it, or lies behind it."""
    check_gemm(M, K, N, fmt, bias=bias, residual=residual)


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("M,K,N", [(2041, 96, 3400), (1100, 64, 2056), (700, 5152, 392)])
def test_gemm_tiles_in_place(M, K, N, fmt):
    """residual is y, over many tiles of a pair, and where pairs share a tile: a chain of calls, each onto the last one's y."""
    dev = device()
    g = ref.gen(M + N)
    xq, xs, _ = operand(g, M, K, fmt)
    wq, ws, _ = operand(g, N, K, fmt, std=K ** -0.5)
    y = ref.randn(g, M, N).to(dev)
    want = y.clone()
    for _ in range(4):
        want = ck.fp4_gemm(xq, xs, wq, ws, fmt, alpha=T[fmt] ** 2, residual=want)
    for _ in range(4):
        assert ck.fp4_gemm(xq, xs, wq, ws, fmt, alpha=T[fmt] ** 2, residual=y, out=y) is y
    poll_ok()
    assert torch.equal(y, want)


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("M,K,N,bias,residual", [(33, 5152, 200, True, True), (256, 7712, 1032, False, False), (300, 10272, 392, True, False),
                                                 (129, 16384, 2048, False, True), (64, 12288, 4096, True, True), (700, 16416, 328, False, False),
                                                 (513, 8192, 776, True, True)])
def test_gemm_few_tiles_long_k(M, K, N, fmt, bias, residual):
    """K divided between the pairs of a cluster, two, three and four of them."""
    check_gemm(M, K, N, fmt, bias=bias, residual=residual)


@pytest.mark.parametrize("fmt", FMTS)
def test_gemm_long_k_in_place_and_nan(fmt):
    dev = device()
    g = ref.gen(77)
    M, K, N = 70, 10240, 264
    x = ref.randn(g, M, K).to(dev)
    x[40, 9000] = float("inf")  # of the last share of K
    xq, xs = ck.fp4_quantize(x, fmt, scale=T[fmt])
    wq, ws = ck.fp4_quantize(ref.randn(g, N, K, std=K ** -0.5).to(dev), fmt, scale=T[fmt])
    r = ref.randn(g, M, N).to(dev)
    want = ck.fp4_gemm(xq, xs, wq, ws, fmt, alpha=T[fmt] ** 2, residual=r)
    for _ in range(20):  # the same bits every time
        again = ck.fp4_gemm(xq, xs, wq, ws, fmt, alpha=T[fmt] ** 2, residual=r)
        assert torch.equal(again.nan_to_num(), want.nan_to_num())
    got = ck.fp4_gemm(xq, xs, wq, ws, fmt, alpha=T[fmt] ** 2, residual=r, out=r)
    poll_ok()
    assert got is r and torch.equal(got.isnan(), want.isnan()) and torch.equal(got.nan_to_num(), want.nan_to_num())
    assert bool(want[40].isnan().all()) and not bool(want[:40].isnan().any()) and not bool(want[41:].isnan().any())


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("M", [4, 40, 400])
def test_gemm_nan_scales(M, fmt):
    """A block with a NaN scale makes its row of X, or its row of W, NaN, and nothing else."""
    dev = device()
    g = ref.gen(M)
    K, N = 224, 200
    out = []
    for rows in (M, N):
        codes, scales = ref.quantize(ref.randn(g, rows, K, dtype=torch.float32).numpy(), fmt, T[fmt])
        scales[rows // 2, 3] = 255 if fmt == "mx" else 0x7f
        out.append((torch.from_numpy(ref.pack(codes)).to(dev), torch.from_numpy(ref.tile(scales, fmt)).to(dev), ref.values(codes, scales, fmt)))
    (xq, xs, xv), (wq, ws, wv) = out
    y = ck.fp4_gemm(xq, xs, wq, ws, fmt, alpha=0.25).float().cpu().numpy()
    poll_ok()
    bad = np.zeros((M, N), bool)
    bad[M // 2], bad[:, N // 2] = True, True
    assert np.array_equal(np.isnan(y), bad)
    want, bound = ref.product(np.nan_to_num(xv), np.nan_to_num(wv), 0.25)
    ref.assert_product(np.where(bad, 0, y), np.where(bad, 0, want), bound)


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("M", [6, 300])
def test_gemm_in_place_residual(M, fmt):
    dev = device()
    g = ref.gen(77)
    xq, xs, _ = operand(g, M, 256, fmt)
    wq, ws, _ = operand(g, 176, 256, fmt)
    r = ref.randn(g, M, 176).to(dev)
    want = ck.fp4_gemm(xq, xs, wq, ws, fmt, alpha=-0.5, residual=r)
    got = ck.fp4_gemm(xq, xs, wq, ws, fmt, alpha=-0.5, residual=r, out=r)
    assert got is r and torch.equal(got, want)
    poll_ok()


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("M,K,N,act", [(1, 32, 8, "none"), (3, 352, 136, "none"), (5, 256, 1032, "swiglu"), (13, 2048, 264, "none"),
                                       (20, 96, 72, "swiglu"), (70, 512, 264, "none"), (600, 672, 392, "swiglu")])
def test_linear_is_quantize_and_product(M, K, N, act, fmt):
    dev = device()
    g = ref.gen(M + N)
    x = ref.randn(g, M, (2 if act == "swiglu" else 1) * K, std=1.5).to(dev)
    w = ref.randn(g, N, K, std=K ** -0.5, dtype=torch.float32).to(dev)
    bias, res = ref.randn(g, N).to(dev), ref.randn(g, M, N).to(dev)
    xt, wt = (1.0, 1.0) if fmt == "mx" else (0.004, 0.0003)
    wq, ws = ck.fp4_quantize(w, fmt, scale=wt)
    y = ck.fp4_linear(x, wq, ws, fmt, x_scale=xt, w_scale=wt, bias=bias, act=act, residual=res)
    xq, xs = ck.fp4_quantize(x, fmt, scale=xt, act=act)
    codes, scales = ref.unpack(xq.cpu().numpy()), ref.untile(xs.cpu().numpy(), M, K, fmt)
    wc, wsc = ref.unpack(wq.cpu().numpy()), ref.untile(ws.cpu().numpy(), N, K, fmt)
    alpha = float(np.float32(np.float32(xt) * np.float32(wt)))
    want, bound = ref.product(ref.values(codes, scales, fmt), ref.values(wc, wsc, fmt), alpha, bias.double().cpu().numpy(),
                              res.double().cpu().numpy())
    ref.assert_product(y, want, bound)
    assert torch.equal(y, ck.fp4_linear(x, wq, ws, fmt, x_scale=xt, w_scale=wt, bias=bias, act=act, residual=res))
    poll_ok()


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("M", [1, 5, 16, 100, 500])
def test_linear_in_place_and_rows_apart(M, fmt):
    """x is a view of wider rows; x, residual and y are one tensor."""
    dev = device()
    g = ref.gen(M)
    K = 320
    wide = ref.randn(g, M, 3 * K).to(dev)
    x = wide[:, K:2 * K]
    wq, ws = ck.fp4_quantize(ref.randn(g, K, K, std=K ** -0.5).to(dev), fmt, scale=T[fmt])
    kw = dict(x_scale=T[fmt], w_scale=T[fmt])
    plain = ck.fp4_linear(x.contiguous(), wq, ws, fmt, **kw)
    assert torch.equal(ck.fp4_linear(x, wq, ws, fmt, **kw), plain)
    z = x.contiguous()
    want = ck.fp4_linear(z.clone(), wq, ws, fmt, residual=z.clone(), **kw)
    assert torch.equal(ck.fp4_linear(z, wq, ws, fmt, residual=z, out=z, **kw), want)
    poll_ok()


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("M,H,I", [(1, 96, 64), (6, 512, 1056), (40, 256, 352), (300, 224, 544)])
def test_mlp_is_two_linears(M, H, I, fmt):
    dev = device()
    g = ref.gen(M + H)
    x = ref.randn(g, M, H).to(dev)
    t = [1.0] * 4 if fmt == "mx" else [0.004, 0.0005, 0.003, 0.0006]
    gu = ck.fp4_quantize(ref.randn(g, 2 * I, H, std=H ** -0.5).to(dev), fmt, scale=t[1])
    d = ck.fp4_quantize(ref.randn(g, H, I, std=I ** -0.5).to(dev), fmt, scale=t[3])
    bgu, bd = ref.randn(g, 2 * I, std=0.1).to(dev), ref.randn(g, H, std=0.1).to(dev)
    y = ck.fp4_swiglu_mlp(x, *gu, *d, fmt, x_scale=t[0], gate_up_scale=t[1], act_scale=t[2], down_scale=t[3], bgu=bgu, bd=bd,
                          residual=x)
    h = ck.fp4_linear(x, *gu, fmt, x_scale=t[0], w_scale=t[1], bias=bgu)
    want = ck.fp4_linear(h, *d, fmt, x_scale=t[2], w_scale=t[3], bias=bd, act="swiglu", residual=x)
    assert torch.equal(y, want)
    z = x.clone()
    ck.fp4_swiglu_mlp(z, *gu, *d, fmt, x_scale=t[0], gate_up_scale=t[1], act_scale=t[2], down_scale=t[3], bgu=bgu, bd=bd,
                      residual=z, out=z)
    assert torch.equal(z, want)
    poll_ok()


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("M,H,I", [(33, 96, 64), (129, 544, 192), (257, 256, 576), (300, 1056, 320), (600, 512, 1088), (1000, 256, 3008)])
def test_mlp_gate_and_up_on_chip(M, H, I, fmt):
    """Where I is a multiple of 64 the first product quantizes silu(gate) * up itself: the same bits as two linears, its
    scales' missing blocks too (the second product would show them)."""
    test_mlp_is_two_linears(M, H, I, fmt)


@pytest.mark.parametrize("fmt", FMTS)
def test_mlp_not_finite(fmt):
    """A token with a NaN, and a gate row with one, stay with their rows; an infinite gate's silu is its own block's."""
    dev = device()
    g = ref.gen(8)
    M, H, I = 70, 256, 192
    x = ref.randn(g, M, H)
    x[5, 7] = float("nan")
    t = T[fmt]
    gu = ck.fp4_quantize(ref.randn(g, 2 * I, H, std=H ** -0.5).to(dev), fmt, scale=t)
    d = ck.fp4_quantize(ref.randn(g, H, I, std=I ** -0.5).to(dev), fmt, scale=t)
    kw = dict(x_scale=t, gate_up_scale=t, act_scale=t, down_scale=t)
    y = ck.fp4_swiglu_mlp(x.to(dev), *gu, *d, fmt, **kw)
    h = ck.fp4_linear(x.to(dev), *gu, fmt, x_scale=t, w_scale=t)
    want = ck.fp4_linear(h, *d, fmt, x_scale=t, w_scale=t, act="swiglu")
    poll_ok()
    assert torch.equal(torch.isnan(y), torch.isnan(want)) and torch.isnan(y[5]).all() and not torch.isnan(y[:5]).any()
    assert torch.equal(torch.nan_to_num(y), torch.nan_to_num(want))


@pytest.mark.parametrize("M", [2, 300])
def test_graph_and_streams(M):
    """Captured and replayed on changed inputs; another stream; two graphs that share a workspace, replayed in turn."""
    dev = device()
    fmt, K, N = "nv", 512, 264
    g = ref.gen(5)
    w = ck.fp4_quantize(ref.randn(g, N, K, std=K ** -0.5).to(dev), fmt, scale=0.001)
    a, b = (ref.randn(g, M, K).to(dev) for _ in range(2))
    ws = ck.fp4_linear_workspace(M, K, fmt)
    def call(x, out=None):
        return ck.fp4_linear(x, *w, fmt, x_scale=0.004, w_scale=0.001, out=out, workspace=ws)
    ya, yb = call(a), call(b)
    torch.cuda.synchronize()
    outs, graphs = [torch.empty_like(ya) for _ in range(2)], []
    for x, out in zip((a, b), outs):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            call(x, out)
        graphs.append(graph)
    for i in (0, 1, 0, 1, 1, 0):
        graphs[i].replay()
    torch.cuda.synchronize()
    assert torch.equal(outs[0], ya) and torch.equal(outs[1], yb)
    a.copy_(b)
    graphs[0].replay()
    torch.cuda.synchronize()
    assert torch.equal(outs[0], yb)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    ys = ck.fp4_linear(b, *w, fmt, x_scale=0.004, w_scale=0.001, stream=s)
    s.synchronize()
    assert torch.equal(ys, yb)
    poll_ok()


def test_binding_refuses():
    dev = device()
    x = torch.zeros(4, 64, dtype=torch.bfloat16, device=dev)
    wq, ws = ck.fp4_quantize(torch.ones(16, 64, dtype=torch.bfloat16, device=dev), "mx")
    with pytest.raises(ValueError):
        ck.fp4_linear(x, wq, ws, "fp4")
    with pytest.raises(ValueError):
        ck.fp4_linear(x.cpu(), wq, ws, "mx")
    with pytest.raises(ValueError):
        ck.fp4_linear(x[:, :32], wq, ws, "mx")
    with pytest.raises(ValueError):
        ck.fp4_linear(x.t().contiguous().t(), wq, ws, "mx")
    with pytest.raises(ValueError):
        ck.fp4_linear(x, wq, ws[:100], "mx")
    with pytest.raises(ValueError):
        ck.fp4_linear(x, wq, ws, "mx", bias=torch.zeros(15, dtype=torch.bfloat16, device=dev))
    with pytest.raises(ValueError):
        ck.fp4_linear(x, wq, ws, "mx", residual=torch.zeros(4, 16, device=dev))
    with pytest.raises(ValueError):
        ck.fp4_linear(x, wq, ws, "mx", act="gelu")
    with pytest.raises(ck.CkError):
        ck.fp4_linear(x, wq, ws, "mx", x_scale=0.5)
    with pytest.raises(ck.CkError):
        ck.fp4_linear(x, wq, ws, "mx", workspace=torch.empty(16, dtype=torch.uint8, device=dev))
    with pytest.raises(ck.CkError):
        ck.fp4_quantize(torch.zeros(4, 40, dtype=torch.bfloat16, device=dev), "mx")
    with pytest.raises(ValueError):
        ck.fp4_quantize(torch.zeros(4, 64, dtype=torch.float16, device=dev), "mx")
    poll_ok()
