"""The 4-bit operators and the block norm as a server calls them: captured into graphs
that share a workspace, on several streams at once, with overlapped launches, and over
rows whose offsets pass 32 bits."""
import threading

import pytest
import torch

import fp4_reference as ref
import swiglu_mlp_group_gb300 as ck
from gpu_helpers import device, poll_ok

pytestmark = pytest.mark.gpu

H, I = 256, 576


class Layer:
    """Norm to codes, product, sum and norm, MLP: every output of a layer's calls is kept."""

    def __init__(self, M, fmt, seed):
        dev = device()
        g = ref.gen(seed)
        self.M, self.fmt, self.t = M, fmt, 1.0 if fmt == "mx" else 0.004
        self.x, self.branch = ref.randn(g, M, H).to(dev), ref.randn(g, M, H).to(dev)
        self.mod = ref.randn(g, -(-M // 4), 3 * H, std=0.3).to(dev)
        self.weight = ref.randn(g, H, std=0.1, mean=1.0).to(dev)
        self.w1, self.gu, self.d = (ck.fp4_quantize(ref.randn(g, n, k, std=k ** -0.5).to(dev), fmt, scale=self.t)
                                    for n, k in ((H, H), (2 * I, H), (H, I)))
        self.ws = ck.fp4_swiglu_mlp_workspace(M, H, I, fmt)
        self.out = {name: torch.empty(M, H, dtype=torch.bfloat16, device=dev) for name in ("h", "a", "h2", "n", "y", "z")}
        self.codes, self.scales = ck.fp4_quantize(self.x, fmt, scale=self.t)
        torch.cuda.synchronize()  # the weights are settled

    def __call__(self, stream=None):
        o, t, fmt = self.out, self.t, self.fmt
        m = dict(gate=self.mod[:, :H], scale=self.mod[:, H:2 * H], shift=self.mod[:, 2 * H:], tokens_per_group=4)
        ck.block_norm_fp4(self.x, self.branch, fmt=fmt, n_scale=t, weight=self.weight, norm="layer", h_out=o["h"],
                          codes=self.codes, scales=self.scales, stream=stream, **m)
        ck.fp4_gemm(self.codes, self.scales, *self.w1, fmt, alpha=t * t, out=o["a"], stream=stream)
        ck.block_norm(o["h"], o["a"], weight=self.weight, h_out=o["h2"], n_out=o["n"], stream=stream)
        ck.fp4_swiglu_mlp(o["n"], *self.gu, *self.d, fmt, x_scale=t, gate_up_scale=t, act_scale=t, down_scale=t,
                          residual=o["h2"], out=o["y"], workspace=self.ws, stream=stream)
        ck.fp4_linear(o["y"], *self.w1, fmt, x_scale=t, w_scale=t, residual=o["y"], out=o["z"], workspace=self.ws,
                      stream=stream)

    def result(self):
        torch.cuda.synchronize()
        poll_ok()
        return {k: v.clone() for k, v in self.out.items()}

    def clear(self):
        for v in self.out.values():
            v.fill_(float("nan"))
        torch.cuda.synchronize()


def same(a, b):
    for k in a:
        assert torch.equal(a[k], b[k]), k


SIZES = [(1, "nv"), (8, "mx"), (21, "nv"), (300, "mx"), (300, "nv")]


@pytest.mark.parametrize("M,fmt", SIZES)
def test_overlapped_launches(M, fmt):
    layer = Layer(M, fmt, M)
    layer()
    want = layer.result()
    layer.clear()
    ck.set_launch_overlap(True)
    try:
        for _ in range(5):
            layer()
        same(layer.result(), want)
    finally:
        ck.set_launch_overlap(False)


@pytest.mark.parametrize("M,fmt", SIZES)
def test_graphs(M, fmt):
    """Two layers captured, which share workspace and codes; replayed in turn, and on changed inputs."""
    a, b = Layer(M, fmt, M), Layer(M, fmt, M + 1)
    b.ws, b.codes, b.scales = a.ws, a.codes, a.scales
    want = []
    for layer in (a, b):
        layer()
        want.append(layer.result())
    graphs = []
    for layer in (a, b):
        layer.clear()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            layer()
        graphs.append(graph)
    for i in (0, 1, 1, 0, 0, 1, 0):
        graphs[i].replay()
    same(a.result(), want[0])
    same(b.result(), want[1])
    a.x.copy_(b.x)
    a.branch.copy_(b.branch)
    graphs[0].replay()
    got = a.result()
    a()
    same(got, a.result())
    assert not torch.equal(got["y"], want[0]["y"])


def test_threads_and_streams():
    """Layers of several sizes and both formats at once, a thread and a stream each."""
    layers = [Layer(M, fmt, 50 + i) for i, (M, fmt) in enumerate(SIZES)]
    want = []
    for layer in layers:
        layer()
        want.append(layer.result())
        layer.clear()
    errors = []

    def work(layer):
        try:
            torch.cuda.set_device(0)
            stream = torch.cuda.Stream()
            for _ in range(20):
                layer(stream)
            stream.synchronize()
        except Exception as e:  # noqa: BLE001
            errors.append(e)
    threads = [threading.Thread(target=work, args=(layer,)) for layer in layers]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not errors, errors
    for layer, w in zip(layers, want):
        same(layer.result(), w)


def test_rows_past_32_bits():
    """Rows so far apart that their offsets (elements and bytes) pass 32 bits, against the same rows together."""
    dev = device()
    g = ref.gen(9)
    ld, T, K = (1 << 31) - 8, 3, 64
    far = torch.empty((T - 1) * ld + 2 * K, dtype=torch.bfloat16, device=dev)  # 8.6 GB
    x = far.as_strided((T, 2 * K), (ld, 1))
    near = ref.randn(g, T, 2 * K).to(dev)
    x.copy_(near)
    w = ck.fp4_quantize(ref.randn(g, 64, K).to(dev), "mx")
    for act, cols in (("none", K), ("swiglu", 2 * K)):
        (codes, scales), (want, want_scales) = (ck.fp4_quantize(v[:, :cols], "mx", act=act) for v in (x, near))
        assert torch.equal(codes, want)
        assert (ref.untile(scales.cpu().numpy(), T, K, "mx") == ref.untile(want_scales.cpu().numpy(), T, K, "mx")).all()
        assert torch.equal(ck.fp4_linear(x[:, :cols], *w, "mx", act=act), ck.fp4_linear(near[:, :cols], *w, "mx", act=act))
    h, n = ck.block_norm(near, near)
    hf, nf = ck.block_norm(x, x, h_out=x)
    assert torch.equal(hf, h) and torch.equal(nf, n) and torch.equal(x, h)
    poll_ok()


@pytest.mark.parametrize("residual", [False, True])
def test_output_past_32_bits(residual):
    """y of 4.3 G elements: rows all over it against the product of those rows alone."""
    dev = device()
    M, K, N = 530000, 32, 8192
    g = ref.gen(10)
    x = ref.randn(g, 1000, K).to(dev).repeat(M // 1000, 1)
    wq, ws = ck.fp4_quantize(ref.randn(g, N, K).to(dev), "nv", scale=0.004)
    xq, xs = ck.fp4_quantize(x, "nv", scale=0.004)
    y = torch.empty(M, N, dtype=torch.bfloat16, device=dev)
    if residual:
        y.fill_(3.0)
    ck.fp4_gemm(xq, xs, wq, ws, "nv", alpha=1.6e-5, out=y, residual=y if residual else None)
    part = ck.fp4_quantize(x[:1000], "nv", scale=0.004)
    r = torch.full((1000, N), 3.0, dtype=torch.bfloat16, device=dev) if residual else None
    want = ck.fp4_gemm(*part, wq, ws, "nv", alpha=1.6e-5, residual=r)
    assert float(want.abs().max()) > 0
    for first in range(0, M, 1000):
        assert torch.equal(y[first:first + 1000], want), first
    poll_ok()


def test_norm_codes_past_32_bits():
    """4.4 G channels: the last rows' codes and scales against those of the rows alone."""
    dev = device()
    T, K = 270000, 16384
    g = ref.gen(11)
    x = torch.empty(T, K, dtype=torch.bfloat16, device=dev)
    some = ref.randn(g, 128, K).to(dev)
    x[-128:], x[:128], x[128:-128] = some, some, 0
    assert T % 128 == 48  # those rows lie in two tiles of scales
    want = ck.block_norm_fp4(some, fmt="mx")
    got = ck.block_norm_fp4(x, fmt="mx")
    assert torch.equal(got[1][:128], want[1]) and torch.equal(got[1][-128:], want[1])
    tiles = got[2].view(-1, K // 128, 32, 4, 4)  # [tile, word, row % 32, row / 32, byte]
    by_row = lambda t: t.permute(0, 3, 2, 1, 4).reshape(t.shape[0] * 128, -1)  # noqa: E731
    last = by_row(tiles[-2:])[48:48 + 128]
    first = by_row(want[2].view(-1, K // 128, 32, 4, 4))
    assert torch.equal(last, first) and torch.equal(by_row(tiles[:1]), first)
    poll_ok()
