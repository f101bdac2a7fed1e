"""One decoder layer of a serving step on the library alone: B sequences behind a
shared prompt, each with its own generated tokens in a paged cache.

    x -> qkv (INT8 decode GEMV) -> head norm + position rotation of the queries,
    keys (normed and rotated) and values appended to the cache -> attention over
    the shared prompt and each sequence's own tokens -> output projection + x
    -> SwiGLU MLP + residual

and, where encoder states are given, a cross attention between the two.  The same
layer with its norms, on 4-bit weights (Fp4DecoderLayer): each norm takes in the sum
of the residual stream and the branch ahead, and goes straight to the codes that the
next product reads.  Every step runs in the library's CUDA kernels; torch holds the
memory.

    python examples/decoder_layer.py        # a few steps, checked against float64 attention
"""
import math
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import swiglu_mlp_group_gb300 as ck  # noqa: E402

G = 64  # rotation group of the INT8 weights


class Linear:
    """An INT8 ConvRot weight: GEMV-resident for up to 8 tokens, GEMM-resident beyond."""

    def __init__(self, W):
        self.N = W.shape[0]
        q, self.scale = ck.quantize_weight(W, G)
        self.gemv = ck.prepare_weight(q, self.scale, ck.CK_WLAYOUT_GEMV_PACKED)
        self.gemm = ck.prepare_weight(q, self.scale, ck.CK_WLAYOUT_GEMM_F16)

    def __call__(self, x, residual=None):
        if x.shape[0] <= 8:
            return ck.gemv_smallM(x, self.gemv, self.N, G, residual=residual)
        return ck.int8_linear(x, self.gemm, self.scale, G, wlayout=ck.CK_WLAYOUT_GEMM_F16, residual=residual)


class Fp4Linear:
    """A weight of microscaled 4-bit floats, its scales in the order that the tensor cores read."""

    def __init__(self, W, fmt):
        self.N, self.fmt = W.shape[0], fmt
        # an NV tensor's scale lets its largest block scale reach E4M3's largest number
        self.scale = float(W.abs().max()) / (6 * 448) if fmt == "nv" else 1.0
        self.x_scale = 16 / (6 * 448) if fmt == "nv" else 1.0
        self.W, self.scales = ck.fp4_quantize(W.float(), fmt, scale=self.scale)

    def __call__(self, x, residual=None):
        return ck.fp4_linear(x, self.W, self.scales, self.fmt, x_scale=self.x_scale, w_scale=self.scale,
                             residual=residual)


class DecoderLayer:
    def __init__(self, hidden=512, inner=1024, Hq=8, Hkv=2, D=64, page=16, pages=256, max_pos=4096, seed=0, device="cuda"):
        gen = torch.Generator(device="cpu").manual_seed(seed)

        def weight(n, k):
            return (torch.randn(n, k, generator=gen) / math.sqrt(k)).to(device)

        self.Hq, self.Hkv, self.D, self.page = Hq, Hkv, D, page
        self.qkv = self._linear(weight((Hq + 2 * Hkv) * D, hidden))
        self.out = self._linear(weight(hidden, Hq * D))
        self.cross_q, self.cross_out = self._linear(weight(Hq * D, hidden)), self._linear(weight(hidden, Hq * D))
        self._init_mlp(weight(2 * inner, hidden), weight(hidden, inner))
        self.q_norm = torch.ones(D, dtype=torch.bfloat16, device=device)
        self.k_norm = torch.ones(D, dtype=torch.bfloat16, device=device)
        inv = 10000.0 ** (-torch.arange(0, D, 2, dtype=torch.float64) / D)
        angle = torch.arange(max_pos, dtype=torch.float64)[:, None] * inv
        self.cos_sin = torch.cat([angle.cos(), angle.sin()], 1).float().to(device)
        self.k_cache = torch.zeros(pages, Hkv, page, D, dtype=torch.bfloat16, device=device)
        self.v_cache = torch.zeros_like(self.k_cache)

    def _linear(self, W):
        return Linear(W)

    def _init_mlp(self, gate_up, down):
        gate_up, self.gate_up_scale = ck.quantize_weight(gate_up, G)
        down, self.down_scale = ck.quantize_weight(down, G)
        self.gate_up = ck.prepare_weight(gate_up, self.gate_up_scale, ck.CK_WLAYOUT_GEMM_F16)
        self.down = ck.prepare_weight(down, self.down_scale, ck.CK_WLAYOUT_GEMM_F16)

    def _project(self, x):
        """The packed projection of tokens x to queries, keys and values."""
        return self.qkv(x)

    def _mlp(self, x, branch, projection):
        """projection(branch) added to x, and the MLP behind it."""
        x = projection(branch, residual=x)
        return ck.swiglu_mlp(x, self.gate_up, self.gate_up_scale, self.down, self.down_scale, G,
                             wlayout=ck.CK_WLAYOUT_GEMM_F16, residual=x)

    def _heads(self, x):
        """Queries, keys and values as views of the packed projection of tokens x."""
        T, Hq, H, D = x.shape[0], self.Hq, self.Hkv, self.D
        p = self._project(x)
        return (p[:, :Hq * D].view(T, Hq, D), p[:, Hq * D:(Hq + H) * D].view(T, H, D),
                p[:, (Hq + H) * D:].view(T, H, D))

    def fill(self, x, slots, positions):
        """Keys and values of tokens x into the cache (the shared prompt's prefill)."""
        _, k, v = self._heads(x)
        ck.kv_append(k, v, self.k_cache, self.v_cache, slots, self.cos_sin, positions, wk=self.k_norm)

    def step(self, x, slots, positions, prefix_pages, prefix_len, block_table, seq_lens, max_seq_len, states=None,
             state_lens=None):
        """One token of each of B sequences: x [B, hidden] -> [B, hidden].  seq_lens counts this token."""
        B = x.shape[0]
        q, k, v = self._heads(x)
        ck.kv_append(k, v, self.k_cache, self.v_cache, slots, self.cos_sin, positions, wk=self.k_norm)
        q, _ = ck.qk_norm_rope(q, None, self.cos_sin, positions, wq=self.q_norm)
        a = ck.prefix_attention(q[:, None], self.k_cache, self.v_cache, prefix_pages, prefix_len, block_table,
                                seq_lens, max_seq_len)
        if states is None:
            return self._mlp(x, a.view(B, -1), self.out)
        x = self.out(a.view(B, -1), residual=x)
        sk, sv = states
        cq = self.cross_q(x).view(B, 1, self.Hq, self.D)
        c = ck.cross_attention(cq, sk, sv, kv_lens=state_lens)
        return self._mlp(x, c.view(B, -1), self.cross_out)


class Fp4DecoderLayer(DecoderLayer):
    """The layer on 4-bit weights ("mx" or "nv"), with the norms in front of its projection and its MLP."""

    def __init__(self, fmt, hidden=512, device="cuda", **sizes):
        self.fmt = fmt
        super().__init__(hidden=hidden, device=device, **sizes)
        self.norm_in, self.norm_mlp = (torch.ones(hidden, dtype=torch.bfloat16, device=device) for _ in range(2))

    def _linear(self, W):
        return Fp4Linear(W, self.fmt)

    def _init_mlp(self, gate_up, down):
        self.gate_up, self.down = self._linear(gate_up), self._linear(down)

    def _project(self, x):
        w = self.qkv
        _, codes, scales = ck.block_norm_fp4(x, fmt=self.fmt, n_scale=w.x_scale, weight=self.norm_in)
        return ck.fp4_gemm(codes, scales, w.W, w.scales, self.fmt, alpha=w.x_scale * w.scale)

    def _mlp(self, x, branch, projection):
        gu, d = self.gate_up, self.down
        h, n = ck.block_norm(x, projection(branch), weight=self.norm_mlp)
        return ck.fp4_swiglu_mlp(n, gu.W, gu.scales, d.W, d.scales, self.fmt, x_scale=gu.x_scale,
                                 gate_up_scale=gu.scale, act_scale=d.x_scale, down_scale=d.scale, residual=h)


def run(B=4, prompt=150, steps=5, with_states=True, device="cuda", fmt=None):
    """A few steps of a batch behind a shared prompt, on INT8 weights or 4-bit ones (fmt "mx", "nv") -> (attention
    error of the last step, output)."""
    layer = DecoderLayer(device=device) if fmt is None else Fp4DecoderLayer(fmt, device=device)
    gen = torch.Generator(device="cpu").manual_seed(1)
    hidden = layer.out.N

    def tokens(n):
        return torch.randn(n, hidden, generator=gen).to(torch.bfloat16).to(device)

    page = layer.page
    npre = -(-prompt // page)
    prefix_pages = torch.arange(npre, dtype=torch.int32, device=device)
    layer.fill(tokens(prompt), torch.arange(prompt, device=device), torch.arange(prompt, dtype=torch.int32, device=device))
    per = -(-steps // page)
    block_table = (npre + torch.arange(B * per, dtype=torch.int32, device=device)).view(B, per)
    states = None
    lens = None
    if with_states:
        kv = torch.randn(B, 40, 2 * layer.Hkv * layer.D, generator=gen).to(torch.bfloat16).to(device)
        n = layer.Hkv * layer.D
        states = kv[:, :, :n].view(B, 40, layer.Hkv, layer.D), kv[:, :, n:].view(B, 40, layer.Hkv, layer.D)
        lens = torch.arange(40, 40 - B, -1, dtype=torch.int32, device=device)
    for s in range(steps):
        x = tokens(B)
        slots = block_table[:, s // page].long() * page + s % page
        positions = torch.full((B,), prompt + s, dtype=torch.int32, device=device)
        seq_lens = torch.full((B,), s + 1, dtype=torch.int32, device=device)
        y = layer.step(x, slots, positions, prefix_pages, prompt, block_table, seq_lens, steps, states, lens)
    # the last step's attention again, from the cache in float64
    q, _, _ = layer._heads(x)
    q, _ = ck.qk_norm_rope(q, None, layer.cos_sin, positions, wq=layer.q_norm)
    got = ck.prefix_attention(q[:, None], layer.k_cache, layer.v_cache, prefix_pages, prompt, block_table, seq_lens, steps)
    worst = 0.0
    for b in range(B):
        def rows(cache):
            shared = cache[prefix_pages.long()].transpose(0, 1).flatten(1, 2)[:, :prompt]
            own = cache[block_table[b].long()].transpose(0, 1).flatten(1, 2)[:, :steps]
            return torch.cat([shared, own], 1).double().repeat_interleave(layer.Hq // layer.Hkv, 0)
        p = torch.softmax(torch.einsum("hd,hnd->hn", q[b].double(), rows(layer.k_cache)) / math.sqrt(layer.D), -1)
        want = torch.einsum("hn,hnd->hd", p, rows(layer.v_cache))
        worst = max(worst, float((got[b, 0].double() - want).norm() / want.norm()))
    if ck.poll_device_status() != ck.CK_OK:
        raise RuntimeError("the device status reports a fault")
    return worst, y


if __name__ == "__main__":
    ck.build()
    for fmt in (None, "mx", "nv"):
        error, y = run(fmt=fmt)
        print(f"{fmt or 'int8'} weights: attention of the last step: relative error {error:.2e} against float64; "
              f"layer output {tuple(y.shape)}, finite: {bool(torch.isfinite(y.float()).all())}")
