"""Many query tokens over short states: whole items of one to three key tiles, many
of them to a CTA, among them runs of sequences that have none.  Their results
leave through the ring of K and V tiles, and with so few tiles an item the roles
of the kernel can be several items apart."""
import pytest
import torch

import attention_reference as ref
import swiglu_mlp_group_gb300 as ck
from gpu_helpers import device, poll_ok

pytestmark = pytest.mark.gpu


def some(kind, B, Lk):
    if kind == "all":
        return [Lk] * B
    if kind == "ragged":
        return [(Lk * (3 * b + 2)) // (3 * B) + 1 for b in range(B)]
    return [Lk if b % 4 == 0 else 0 for b in range(B)]  # runs of none


def check(q, k, v, lens):
    B, Lq, Hq, D = q.shape
    out = ck.cross_attention(q, k, v, kv_lens=torch.tensor(lens, dtype=torch.int32, device=q.device))
    poll_ok()
    want, mag = ref.attend(q, [k[b, :lens[b]] for b in range(B)], [v[b, :lens[b]] for b in range(B)],
                           [[lens[b]] * Lq for b in range(B)], D ** -0.5)
    ref.assert_attention(out, want, mag, f"B{B} Lq{Lq} {Hq}x{D} lens {lens[:8]}")


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("Lk", [77, 150, 333])
@pytest.mark.parametrize("B,H", [(2, 16), (8, 6)])
@pytest.mark.parametrize("kind", ["all", "ragged", "runs of none"])
def test_short_states(kind, B, H, Lk, D):
    dev = device()
    g = torch.Generator(device=dev)
    g.manual_seed(B + Lk + D)

    def randn(n, std):
        return (torch.randn(B, n, H, D, generator=g, device=dev) * std).to(torch.bfloat16)

    check(randn(4096, 1.5), randn(Lk, 1.0), randn(Lk, 1.0), some(kind, B, Lk))


# three short sequences, forty of none and many long ones, in shares by cost: the
# CTA that has the first three looks at all those of none before it goes on
LENGTHS = [100] * 3 + [0] * 40 + [4300] * 157


@pytest.mark.parametrize("D", [64, 128])
def test_short_items_before_many_empty_sequences(D):
    dev = device()
    g = torch.Generator(device=dev)
    g.manual_seed(D)
    B = len(LENGTHS)
    q = (torch.randn(B, 200, 1, D, generator=g, device=dev) * 1.5).to(torch.bfloat16)
    k, v = (torch.randn(B, 4300, 1, D, generator=g, device=dev).to(torch.bfloat16) for _ in range(2))
    check(q, k, v, LENGTHS)


@pytest.mark.parametrize("D", [64, 128])
def test_short_items_before_many_empty_sequences_paged(D):
    dev = device()
    B = len(LENGTHS)
    c = ref.Paged(40, B, 1, D, 128, 0, LENGTHS, junk=float("nan")).to(dev)
    q = ref.randn(ref.gen(41), B, 200, 1, D, std=1.5).to(dev)
    out = ck.prefix_attention(q, c.k_cache, c.v_cache, None, 0, c.block_table, c.seq_lens, c.max_len)
    poll_ok()
    want, mag = c.reference(q, D ** -0.5)
    ref.assert_attention(out, want, mag)
