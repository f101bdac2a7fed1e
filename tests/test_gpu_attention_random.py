"""Attention at random sizes: every way of cutting the work (whole groups, fixed
chunks, shares by cost), wide and narrow items in one call, lengths from none to
the longest, against the definition in 64 bits."""
import random

import pytest
import torch

import attention_reference as ref
import swiglu_mlp_group_gb300 as ck
from gpu_helpers import device, poll_ok

pytestmark = pytest.mark.gpu


def lengths(rng, B, top):
    kind = rng.choice(["spread", "one long", "few", "equal"])
    if kind == "one long":
        return [top if b == B // 2 else 0 for b in range(B)]
    if kind == "few":
        return [rng.choice([0, 0, 0, 1, top]) for _ in range(B)]
    if kind == "equal":
        return [top] * B
    return [rng.randint(0, top) for _ in range(B)]


@pytest.mark.parametrize("seed", range(30))
def test_prefix_random(seed):
    dev = device()
    rng = random.Random(seed)
    D, page = rng.choice([64, 128]), rng.choice([16, 32, 64, 128])
    H = rng.choice([1, 2, 3, 4])
    G = rng.choice([1, 2, 3, 5, 8, 16])
    B = rng.choice([1, 3, 17, 60, 150])
    Lq = rng.choice([1, 1, 1, 2, 7, 70])
    if B * Lq > 400:
        Lq = 1
    prefix = rng.choice([0, 1, 130, 700, 2500])
    top = rng.choice([0, 1, 40, 200, 900, 3000])
    if B * top > 60000:
        top = 60000 // B
    lens = lengths(rng, B, top)
    c = ref.Paged(seed, B, H, D, page, prefix, lens, max_len=top + rng.choice([0, 5, 500])).to(dev)
    q = ref.randn(ref.gen(seed + 100), B, Lq, H * G, D, std=1.5).to(dev)
    out = ck.prefix_attention(q, c.k_cache, c.v_cache, c.prefix_pages, c.prefix_len, c.block_table, c.seq_lens, c.max_len)
    poll_ok()
    want, mag = c.reference(q, D ** -0.5)
    ref.assert_attention(out, want, mag, f"B{B} Lq{Lq} {H * G}/{H}x{D} page {page} prefix {prefix} lens {lens}")
    again = ck.prefix_attention(q, c.k_cache, c.v_cache, c.prefix_pages, c.prefix_len, c.block_table, c.seq_lens, c.max_len)
    assert torch.equal(out, again)


@pytest.mark.parametrize("seed", range(20))
def test_cross_random(seed):
    dev = device()
    rng = random.Random(1000 + seed)
    D, H, G = rng.choice([64, 128]), rng.choice([1, 2, 6]), rng.choice([1, 2, 3, 8])
    B, Lq, Lk = rng.choice([1, 2, 9, 40]), rng.choice([1, 5, 63, 200, 700]), rng.choice([1, 77, 300, 1200, 4000])
    while B * Lq * Lk * H * G > 3e8:
        Lk = max(1, Lk // 2)
        B = max(1, B // 2)
    lens = [min(n, Lk) for n in lengths(rng, B, Lk)]
    g = ref.gen(seed + 2000)
    q = ref.randn(g, B, Lq, H * G, D, std=1.5).to(dev)
    kv = ref.randn(g, B, Lk, 2 * H * D)
    for b in range(B):
        kv[b, lens[b]:] = float("nan")
    kv = kv.to(dev)
    k, v = kv[:, :, :H * D].view(B, Lk, H, D), kv[:, :, H * D:].view(B, Lk, H, D)
    out = ck.cross_attention(q, k, v, kv_lens=torch.tensor(lens, dtype=torch.int32, device=dev))
    poll_ok()
    want, mag = ref.attend(q, [k[b, :lens[b]] for b in range(B)], [v[b, :lens[b]] for b in range(B)],
                           [[lens[b]] * Lq for b in range(B)], D ** -0.5)
    ref.assert_attention(out, want, mag, f"B{B} Lq{Lq} Lk{Lk} {H * G}/{H}x{D} lens {lens}")
