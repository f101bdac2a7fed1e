"""One decoder layer of a serving step on the library alone: B sequences behind a
shared prompt, each with its own generated tokens in a paged cache.

    x -> qkv (INT8 decode GEMV) -> head norm + position rotation of the queries,
    keys (normed and rotated) and values appended to the cache -> attention over
    the shared prompt and each sequence's own tokens -> output projection + x
    -> SwiGLU MLP + residual

and, where encoder states are given, a cross attention between the two.  Every
step runs in the library's CUDA kernels; torch holds the memory.

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


class DecoderLayer:
    def __init__(self, hidden=512, inner=1024, Hq=8, Hkv=2, D=64, page=16, pages=256, max_pos=4096, seed=0, device="cuda"):
        gen = torch.Generator(device="cpu").manual_seed(seed)

        def weight(n, k):
            return (torch.randn(n, k, generator=gen) / math.sqrt(k)).to(device)

        self.Hq, self.Hkv, self.D, self.page = Hq, Hkv, D, page
        self.qkv = Linear(weight((Hq + 2 * Hkv) * D, hidden))
        self.out = Linear(weight(hidden, Hq * D))
        self.cross_q, self.cross_out = Linear(weight(Hq * D, hidden)), Linear(weight(hidden, Hq * D))
        gate_up, self.gate_up_scale = ck.quantize_weight(weight(2 * inner, hidden), G)
        down, self.down_scale = ck.quantize_weight(weight(hidden, inner), G)
        self.gate_up = ck.prepare_weight(gate_up, self.gate_up_scale, ck.CK_WLAYOUT_GEMM_F16)
        self.down = ck.prepare_weight(down, self.down_scale, ck.CK_WLAYOUT_GEMM_F16)
        self.q_norm = torch.ones(D, dtype=torch.bfloat16, device=device)
        self.k_norm = torch.ones(D, dtype=torch.bfloat16, device=device)
        inv = 10000.0 ** (-torch.arange(0, D, 2, dtype=torch.float64) / D)
        angle = torch.arange(max_pos, dtype=torch.float64)[:, None] * inv
        self.cos_sin = torch.cat([angle.cos(), angle.sin()], 1).float().to(device)
        self.k_cache = torch.zeros(pages, Hkv, page, D, dtype=torch.bfloat16, device=device)
        self.v_cache = torch.zeros_like(self.k_cache)

    def _heads(self, x):
        """Queries, keys and values as views of the packed projection of tokens x."""
        T, Hq, H, D = x.shape[0], self.Hq, self.Hkv, self.D
        p = self.qkv(x)
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
        x = self.out(a.view(B, -1), residual=x)
        if states is not None:
            sk, sv = states
            cq = self.cross_q(x).view(B, 1, self.Hq, self.D)
            x = self.cross_out(ck.cross_attention(cq, sk, sv, kv_lens=state_lens).view(B, -1), residual=x)
        return ck.swiglu_mlp(x, self.gate_up, self.gate_up_scale, self.down, self.down_scale, G,
                             wlayout=ck.CK_WLAYOUT_GEMM_F16, residual=x)


def run(B=4, prompt=150, steps=5, with_states=True, device="cuda"):
    """A few steps of a batch behind a shared prompt -> (attention error of the last step, output)."""
    layer = DecoderLayer(device=device)
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
    error, y = run()
    print(f"attention of the last step: relative error {error:.2e} against float64; layer output {tuple(y.shape)}, "
          f"finite: {bool(torch.isfinite(y.float()).all())}")
