"""Values that are not finite where some queries see them and others do not: a token
of a sequence that only the later ones of its query tokens see."""
import math

import pytest
import torch

import attention_reference as ref
import swiglu_mlp_group_gb300 as ck
from gpu_helpers import device, poll_ok

pytestmark = pytest.mark.gpu


def check(seed, Lq, Hq, H, D, page, prefix, lens, bad, keys=False):
    """`bad`: (sequence, tokens back from its last, key head, column, value), put into V, or into K if `keys`."""
    dev = device()
    B = len(lens)
    c = ref.Paged(seed, B, H, D, page, prefix, lens)
    at = []
    for b, back, h, d, value in bad:
        t = lens[b] - 1 - back
        (c.k if keys else c.v)[b][t, h, d] = value
        at.append((b, t, h, d))
    for b in range(B):
        c._fill([p for p in c.block_table[b].tolist() if p >= 0], c.k[b], c.v[b])
    c.to(dev)
    q = ref.randn(ref.gen(seed + 1), B, Lq, Hq, D, std=1.5).to(dev)
    out = ck.prefix_attention(q, c.k_cache, c.v_cache, c.prefix_pages, prefix, c.block_table, c.seq_lens, c.max_len)
    again = ck.prefix_attention(q, c.k_cache, c.v_cache, c.prefix_pages, prefix, c.block_table, c.seq_lens, c.max_len)
    poll_ok()
    assert torch.equal(out.view(torch.int16), again.view(torch.int16))
    # what a query sees of them: its column of V, or the whole row through its score
    hit = torch.zeros(out.shape, dtype=torch.bool, device=dev)
    G = Hq // H
    for b, t, h, d in at:
        first = max(0, t - (lens[b] - Lq))  # the first query token that sees token t
        cols = slice(None) if keys else d
        hit[b, first:, h * G:(h + 1) * G, cols] = True
    assert hit.any() and not hit.all()
    assert not torch.isfinite(out[hit]).any()
    # the others: as if nothing were there
    for b, t, h, d in at:
        (c.k if keys else c.v)[b][t, h, d] = 0
    want, mag = c.reference(q, D ** -0.5)
    got = torch.where(hit, want, out.double())
    if keys:  # a row that does not see the token does not see its key's 0 either
        assert not (got != got).any()
    ref.assert_attention(got, want, mag, f"Lq{Lq} {Hq}/{H}x{D} page {page} prefix {prefix} lens {lens}")


NAN, INF = math.nan, math.inf


# few rows, a narrow tile, a wide one, two row tiles; whole and in parts; one tile of keys and many
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("prefix", [0, 90, 700])
@pytest.mark.parametrize("Lq,Hq,H", [(2, 2, 2), (5, 6, 2), (8, 4, 2), (17, 8, 2), (40, 3, 1), (64, 4, 1), (200, 2, 2),
                                     (300, 4, 2)])
def test_values_that_later_tokens_see(Lq, Hq, H, prefix, D):
    lens = [Lq, Lq + 140, Lq + 1, Lq + 700]
    bad = [(0, 0, 0, 3, NAN), (1, Lq // 2, H - 1, D - 1, INF), (1, 0, 0, 17, -INF), (1, Lq - 2, H - 1, 8, NAN),
           (3, (Lq - 1) // 3, 0, 40, NAN), (3, 0, 0, 40, INF)]
    check(Lq + prefix, Lq, Hq, H, D, 16, prefix, lens, bad)


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("Lq,Hq,H", [(5, 6, 2), (40, 3, 1), (300, 4, 2)])
def test_keys_that_later_tokens_see(Lq, Hq, H, D):
    lens = [Lq, Lq + 140, Lq + 1]
    check(Lq, Lq, Hq, H, D, 32, 90, lens, [(0, 0, 0, 3, NAN), (1, Lq // 2, H - 1, 5, NAN)], keys=True)


# many sequences in turn on every CTA, most with something to note
@pytest.mark.parametrize("Lq,Hq,H", [(3, 4, 2), (20, 6, 2), (130, 2, 1)])
@pytest.mark.parametrize("prefix", [0, 200])
def test_one_item_after_the_other(Lq, Hq, H, prefix):
    lens = [Lq + (61 * b) % 500 for b in range(200)]
    bad = [(b, (5 * b) % (Lq - 1), b % H, (7 * b) % 128, [NAN, INF, -INF][b % 3]) for b in range(200) if b % 5]
    check(7, Lq, Hq, H, 128, 64, prefix, lens, bad)


def test_a_whole_token_and_whole_columns():
    """All columns of a token; and a column in every token that not all see."""
    Lq, D = 70, 64
    lens = [Lq + 300, Lq]
    bad = [(0, 9, 0, d, NAN) for d in range(D)] + [(1, t, 0, 5, INF) for t in range(Lq - 1)]
    check(9, Lq, 3, 1, D, 128, 40, lens, bad)


# the prompt's own attention: long, several row tiles, none of them seeing the last tokens but the last
@pytest.mark.parametrize("D", [64, 128])
def test_prompt(D):
    bad = [(0, 0, 0, 1, NAN), (0, 700, 1, 2, INF), (0, 1300, 0, 63, NAN), (1, 3, 1, 0, NAN)]
    check(11, 1500, 8, 2, D, 64, 0, [1500, 1900], bad)
