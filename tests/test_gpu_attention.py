"""Attention over a paged cache with a shared prefix, and over an encoder's
states, against their definitions in 64 bits."""
import math

import pytest
import torch

import attention_reference as ref
import swiglu_mlp_group_gb300 as ck
from gpu_helpers import device, poll_ok

pytestmark = pytest.mark.gpu

NAN = float("nan")


def run_prefix(c, q, **kw):
    return ck.prefix_attention(q, c.k_cache, c.v_cache, c.prefix_pages, c.prefix_len, c.block_table, c.seq_lens,
                               c.max_len, **kw)


def check_prefix(seed, B, Lq, Hq, H, D, page, prefix, lens, junk=NAN, scale=None, std=1.0, max_len=None):
    dev = device()
    c = ref.Paged(seed, B, H, D, page, prefix, lens, junk=junk, std=std, max_len=max_len).to(dev)
    q = ref.randn(ref.gen(seed + 1), B, Lq, Hq, D, std=1.5).to(dev)
    out = run_prefix(c, q, scale=scale)
    want, mag = c.reference(q, D ** -0.5 if scale is None else scale)
    poll_ok()
    ref.assert_attention(out, want, mag, f"B{B} Lq{Lq} {Hq}/{H}x{D} page {page} prefix {prefix} lens {lens}")
    return out


# one token a sequence: prefixes and lengths about the tile and page edges, pages of every size
@pytest.mark.parametrize("page", [16, 32, 64, 128])
@pytest.mark.parametrize("prefix", [0, 1, 127, 128, 129, 1000])
@pytest.mark.parametrize("D", [64, 128])
def test_prefix_lengths(page, prefix, D):
    check_prefix(prefix + page, 6, 1, 8, 2, D, page, prefix, [0, 1, 15, 128, 130, 300])


# heads: none shared, odd groups, one key head, a whole tile of query heads
@pytest.mark.parametrize("Hq,H", [(1, 1), (5, 5), (6, 2), (10, 2), (7, 1), (24, 4), (32, 8), (128, 1)])
@pytest.mark.parametrize("Lq", [1, 3])
def test_prefix_head_layouts(Hq, H, Lq):
    check_prefix(Hq, 3, Lq, Hq, H, 64, 16, 200, [3, 77, 129])


# several query tokens: causal among a sequence's own; fewer cached tokens than queries leaves early ones without
@pytest.mark.parametrize("Lq", [2, 5, 31, 64, 200])
@pytest.mark.parametrize("prefix", [0, 90])
@pytest.mark.parametrize("D", [64, 128])
def test_prefix_several_queries(Lq, prefix, D):
    check_prefix(Lq, 3, Lq, 6, 2, D, 32, prefix, [1, Lq, Lq + 140])


# many rows against the prefix: more than one tile of them, ragged last tile
@pytest.mark.parametrize("B,Hq,H", [(33, 8, 1), (65, 4, 1), (70, 12, 2), (300, 2, 1)])
@pytest.mark.parametrize("prefix", [513, 2048])
def test_prefix_many_rows(B, Hq, H, prefix):
    check_prefix(B, B, 1, Hq, H, 128, 64, prefix, [(7 * b) % 150 for b in range(B)])


@pytest.mark.parametrize("D", [64, 128])
def test_prefix_long(D):
    check_prefix(11, 4, 1, 8, 2, D, 64, 9001, [4097, 0, 5, 2500])


@pytest.mark.parametrize("junk", [NAN, math.inf, -math.inf, torch.finfo(torch.bfloat16).min])
def test_prefix_unused_rows_do_not_matter(junk):
    a = check_prefix(5, 3, 2, 8, 2, 128, 16, 70, [2, 33, 150], junk=junk)
    b = check_prefix(5, 3, 2, 8, 2, 128, 16, 70, [2, 33, 150], junk=0.0)
    assert torch.equal(a, b)


def test_prefix_empty_rows_are_zero():
    out = check_prefix(6, 3, 2, 8, 2, 64, 16, 0, [0, 1, 40])
    assert (out[0] == 0).all()          # nothing cached
    assert (out[1, 0] == 0).all()       # one cached token, two queries: the first sees none
    assert (out[1, 1] != 0).any()


def test_prefix_all_lengths_zero():
    dev = device()
    c = ref.Paged(7, 2, 2, 128, 16, 100, [0, 0]).to(dev)
    q = ref.randn(ref.gen(8), 2, 1, 4, 128).to(dev)
    out = ck.prefix_attention(q, c.k_cache, c.v_cache, c.prefix_pages, 100, None, None, 0)
    want, mag = c.reference(q, 128 ** -0.5)
    ref.assert_attention(out, want, mag)
    none = ck.prefix_attention(q, c.k_cache, c.v_cache, None, 0, None, None, 0)
    poll_ok()
    assert (none == 0).all()


def test_prefix_large_scores():
    """Scores of hundreds: the running maximum moves far and late, weights of most keys vanish."""
    dev = device()
    c = ref.Paged(9, 2, 1, 64, 16, 700, [30, 300], std=8.0).to(dev)
    q = ref.randn(ref.gen(10), 2, 2, 4, 64, std=8.0).to(dev)
    out = run_prefix(c, q)
    want, mag = c.reference(q, 64 ** -0.5)
    poll_ok()
    # scores of s units are off by s 2^-22 at least, here some 2^-13: covered by the bound's f32 part doubled
    got, bound = out.double(), ref.U * (1 + ref.U) * (mag + want.abs()) + 2.0 ** -11 * mag + 1e-30
    assert ((got - want).abs() <= bound).all()


def test_prefix_growing_scores():
    """Every key beats all before it: the sums are rescaled again and again."""
    dev = device()
    c = ref.Paged(12, 1, 1, 128, 16, 600, [300])
    ramp = torch.linspace(0, 6, 600)[:, None, None]
    c.pk = ramp.expand(600, 1, 128).to(torch.bfloat16)
    c.k[0] = (ramp[:300] + 6).expand(300, 1, 128).to(torch.bfloat16)
    c._fill(c.prefix_pages.tolist(), c.pk, c.pv)
    c._fill(c.block_table[0].tolist(), c.k[0], c.v[0])
    c.to(dev)
    q = torch.ones(1, 1, 2, 128, dtype=torch.bfloat16, device=dev)
    out = run_prefix(c, q)
    want, mag = c.reference(q, 128 ** -0.5)
    poll_ok()
    got, bound = out.double(), ref.U * (1 + ref.U) * (mag + want.abs()) + 2.0 ** -12 * mag + 1e-30
    assert ((got - want).abs() <= bound).all()


def test_prefix_strided_and_given_buffers():
    dev = device()
    B, Lq, Hq, H, D = 3, 2, 6, 2, 64
    c = ref.Paged(13, B, H, D, 32, 150, [2, 60, 140]).to(dev)
    packed = ref.randn(ref.gen(14), B, Lq, (Hq + 2 * H) * D).to(dev)
    q = packed[:, :, :Hq * D].view(B, Lq, Hq, D)
    assert not q.is_contiguous()
    wide = torch.full((B * Lq, Hq * D + 24), 7.0, dtype=torch.bfloat16, device=dev)
    out = wide[:, :Hq * D].view(B, Lq, Hq, D)
    ws = ck.prefix_attention_workspace(q, c.k_cache, c.prefix_len, c.max_len)
    ws.fill_(255)
    got = run_prefix(c, q, out=out, workspace=ws)
    assert got is out and (wide[:, Hq * D:] == 7).all()
    want, mag = c.reference(q, D ** -0.5)
    ref.assert_attention(out, want, mag)
    assert torch.equal(out, run_prefix(c, q))  # the same bits every time, whatever the workspace held
    poll_ok()


def test_prefix_loose_bound_on_lengths():
    """max_seq_len is a bound: lengths may lie far below it."""
    a = check_prefix(15, 4, 1, 8, 2, 128, 16, 300, [3, 0, 17, 90], max_len=4000)
    b = check_prefix(15, 4, 1, 8, 2, 128, 16, 300, [3, 0, 17, 90])
    assert (a.double() - b.double()).abs().max() <= 2.0 ** -6  # other splits, other roundings


def test_prefix_indexes_out_of_range():
    dev = device()
    poll_ok()
    c = ref.Paged(16, 3, 2, 64, 16, 50, [40, 40, 40], junk=0.0).to(dev)
    q = ref.randn(ref.gen(17), 3, 1, 4, 64).to(dev)
    good = run_prefix(c, q)
    poll_ok()
    table = c.block_table.clone()
    c.block_table[1, 0] = c.k_cache.shape[0]
    c.block_table[1, 1] = -1
    out = run_prefix(c, q)
    assert ck.poll_device_status() == ck.CK_ERR_INDEX
    assert ck.poll_device_status() == ck.CK_OK  # cleared on read
    assert torch.equal(out[0], good[0]) and torch.equal(out[2], good[2])
    assert torch.isfinite(out).all()
    c.block_table = table
    for bad, same in ((41, 40), (1 << 30, 40)):  # past max_seq_len: taken as it
        c.seq_lens[1] = bad
        out = run_prefix(c, q)
        assert ck.poll_device_status() == ck.CK_ERR_INDEX
        assert torch.equal(out, good)
    c.seq_lens[1] = -3
    out = run_prefix(c, q)
    assert ck.poll_device_status() == ck.CK_ERR_INDEX
    c.seq_lens[1] = 0
    assert torch.equal(out, run_prefix(c, q))
    poll_ok()


def test_prefix_offsets_past_32_bits():
    """Pages whose elements lie past 2^31 of a long cache; the append that fills them."""
    dev = device()
    D, page, n = 128, 128, 300
    pages = (1 << 31) // (page * D) + 20
    kc = torch.empty(pages, 1, page, D, dtype=torch.bfloat16, device=dev)
    vc = torch.empty_like(kc)
    k, v = ref.randn(ref.gen(18), n, 1, D).to(dev), ref.randn(ref.gen(19), n, 1, D).to(dev)
    mine = torch.tensor([pages - 1, pages - 3, pages - 2], dtype=torch.int32, device=dev)
    t = torch.arange(n, device=dev)
    ck.kv_append(k, v, kc, vc, mine.long()[t // page] * page + t % page)
    q = ref.randn(ref.gen(20), 1, 1, 4, D).to(dev)
    want, mag = ref.attend(q, [k], [v], [[n]], D ** -0.5)
    own = ck.prefix_attention(q, kc, vc, None, 0, mine[None].contiguous(), torch.tensor([n], dtype=torch.int32, device=dev), n)
    ref.assert_attention(own, want, mag)
    shared = ck.prefix_attention(q, kc, vc, mine, n, None, None, 0)
    ref.assert_attention(shared, want, mag)
    poll_ok()


def check_cross(seed, B, Lq, Lk, Hq, H, D, lens, junk=NAN, packed=True):
    dev = device()
    g = ref.gen(seed)
    q = ref.randn(g, B, Lq, Hq, D, std=1.5).to(dev)
    kv = ref.randn(g, B, Lk, 2 * H * D)
    real = [Lk] * B if lens is None else lens
    for b in range(B):
        kv[b, real[b]:] = junk
    kv = kv.to(dev)
    k, v = kv[:, :, :H * D].view(B, Lk, H, D), kv[:, :, H * D:].view(B, Lk, H, D)
    if not packed:
        k, v = k.contiguous(), v.contiguous()
    kl = None if lens is None else torch.tensor(lens, dtype=torch.int32, device=dev)
    out = ck.cross_attention(q, k, v, kv_lens=kl)
    want, mag = ref.attend(q, [k[b, :real[b]] for b in range(B)], [v[b, :real[b]] for b in range(B)],
                           [[real[b]] * Lq for b in range(B)], D ** -0.5)
    poll_ok()
    ref.assert_attention(out, want, mag, f"B{B} Lq{Lq} Lk{Lk} {Hq}/{H}x{D} lens {lens}")
    return out


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("Lk,lens", [(1, [1, 0]), (77, [77, 13]), (128, [128, 127]), (129, [129, 128]),
                                     (333, [200, 333]), (1500, [1500, 257])])
@pytest.mark.parametrize("Lq", [1, 7, 130, 300])
def test_cross_lengths(Lq, Lk, lens, D):
    out = check_cross(Lq + Lk, 2, Lq, Lk, 4, 2, D, lens)
    if 0 in lens:
        assert (out[lens.index(0)] == 0).all()


@pytest.mark.parametrize("Hq,H", [(1, 1), (3, 3), (6, 2), (5, 1), (16, 16), (128, 1)])
@pytest.mark.parametrize("Lq", [1, 50])
def test_cross_head_layouts(Hq, H, Lq):
    check_cross(Hq, 3, Lq, 150, Hq, H, 64, [150, 1, 149])


# up to 16 query rows a key head and just above, and more groups than SMs: every CTA takes several in turn
@pytest.mark.parametrize("Lq,G", [(1, 1), (1, 8), (3, 5), (16, 1), (2, 8), (17, 1), (3, 6)])
@pytest.mark.parametrize("D", [64, 128])
def test_few_rows_many_groups(Lq, G, D):
    lens = [(37 * b) % 700 for b in range(50)]
    check_cross(Lq + G, 50, Lq, 700, 8 * G, 8, D, lens)
    check_prefix(Lq * G, 50, Lq, 2 * G, 2, D, 32, 0, lens)


# scores that grow with the keys, for some rows only: a running maximum that moves in every tile, or in one quarter of it
@pytest.mark.parametrize("Lq", [1, 4, 40])
@pytest.mark.parametrize("every", [1, 37, 128])
@pytest.mark.parametrize("D", [64, 128])
def test_cross_growing_scores(Lq, every, D):
    dev = device()
    B, Lk, H = 3, 1100, 4
    g = ref.gen(Lq + every)
    q, k, v = ref.randn(g, B, Lq, H, D), ref.randn(g, B, Lk, H, D), ref.randn(g, B, Lk, H, D)
    q[:, ::3] = -q[:, ::3]
    # up to 2 sqrt(D): scores whose f32 sums the bound still allows for
    k[:, ::every] = q[:, -1:, :] * torch.linspace(0, 2, Lk)[::every].view(1, -1, 1, 1).to(q.dtype)
    q, k, v = q.to(dev), k.to(dev), v.to(dev)
    out = ck.cross_attention(q, k, v)
    want, mag = ref.attend(q, list(k), list(v), [[Lk] * Lq] * B, D ** -0.5)
    poll_ok()
    ref.assert_attention(out, want, mag)


# more groups than SMs over long states: whole where the lengths are one, in shares where they are not
@pytest.mark.parametrize("B,Lq,Lk,H", [(21, 1, 2300, 8), (23, 20, 2100, 8), (2, 1300, 4300, 14)])
@pytest.mark.parametrize("ragged", [False, True])
@pytest.mark.parametrize("D", [64, 128])
def test_cross_many_groups_long(B, Lq, Lk, H, ragged, D):
    check_cross(B + D, B, Lq, Lk, H, H, D, [(911 * b) % (Lk + 1) for b in range(B - 1)] + [Lk] if ragged else None)


def test_cross_more_rows_than_a_wave():
    check_cross(21, 2, 2500, 300, 6, 3, 128, [300, 299])
    check_cross(22, 1, 1, 5000, 4, 4, 128, None)
    check_cross(23, 40, 1, 40, 4, 4, 64, None, packed=False)


# results into rows of a wider tensor: nothing beside them, before the first or behind the last is written
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("Lq,Hq,H", [(300, 6, 2), (261, 4, 4), (170, 5, 1), (20, 16, 2), (2, 128, 1)])
@pytest.mark.parametrize("Lk", [1, 150, 700])
def test_cross_out_of_wider_rows(Lq, Hq, H, Lk, D):
    dev = device()
    B, wide = 3, Hq * D + 64
    g = ref.gen(Lq + Lk)
    q = ref.randn(g, B, Lq, Hq, D, std=1.5).to(dev)
    k, v = ref.randn(g, B, Lk, H, D).to(dev), ref.randn(g, B, Lk, H, D).to(dev)
    guarded = torch.full((B * Lq + 2, wide), 7.0, dtype=torch.bfloat16, device=dev)
    out = guarded[1:-1, 32:32 + Hq * D].view(B, Lq, Hq, D)
    ck.cross_attention(q, k, v, out=out)
    want, mag = ref.attend(q, list(k), list(v), [[Lk] * Lq] * B, D ** -0.5)
    poll_ok()
    ref.assert_attention(out, want, mag)
    guarded[1:-1, 32:32 + Hq * D] = 7.0
    assert (guarded == 7.0).all()


def test_cross_no_states():
    dev = device()
    q = ref.randn(ref.gen(24), 2, 3, 4, 64).to(dev)
    empty = torch.empty(2, 0, 4, 64, dtype=torch.bfloat16, device=dev)
    out = ck.cross_attention(q, empty, empty)
    poll_ok()
    assert (out == 0).all()


def test_cross_lengths_out_of_range():
    dev = device()
    q = ref.randn(ref.gen(25), 2, 3, 4, 64).to(dev)
    k, v = ref.randn(ref.gen(26), 2, 50, 4, 64).to(dev), ref.randn(ref.gen(27), 2, 50, 4, 64).to(dev)
    good = ck.cross_attention(q, k, v, kv_lens=torch.tensor([50, 0], dtype=torch.int32, device=dev))
    poll_ok()
    out = ck.cross_attention(q, k, v, kv_lens=torch.tensor([51, -1], dtype=torch.int32, device=dev))
    assert ck.poll_device_status() == ck.CK_ERR_INDEX
    assert torch.equal(out, good)


def test_cross_offsets_past_32_bits():
    dev = device()
    Lk, H, D = 1200000, 8, 128  # b = 1 starts 2^31 elements of k and v away with a packed [k | v] row
    kv = torch.empty(2, Lk, 2 * H * D, dtype=torch.bfloat16, device=dev)
    real = ref.randn(ref.gen(28), 2, 40, 2 * H * D).to(dev)
    kv[:, :40] = real
    q = ref.randn(ref.gen(29), 2, 1, 8, D).to(dev)
    out = ck.cross_attention(q, kv[:, :, :H * D].view(2, Lk, H, D), kv[:, :, H * D:].view(2, Lk, H, D),
                             kv_lens=torch.tensor([40, 33], dtype=torch.int32, device=dev))
    n = [40, 33]
    k, v = real[:, :, :H * D].view(2, 40, H, D), real[:, :, H * D:].view(2, 40, H, D)
    want, mag = ref.attend(q, [k[b, :n[b]] for b in range(2)], [v[b, :n[b]] for b in range(2)], [[40], [33]], D ** -0.5)
    ref.assert_attention(out, want, mag)
    poll_ok()


def test_attention_on_another_stream_and_in_a_graph():
    dev = device()
    c = ref.Paged(30, 4, 2, 128, 16, 400, [0, 3, 100, 260]).to(dev)
    q = ref.randn(ref.gen(31), 4, 1, 8, 128).to(dev)
    want = run_prefix(c, q)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    outs = []
    for _ in range(20):  # outputs and workspaces of one call must not be handed out while another still runs
        outs.append(run_prefix(c, q, stream=side))
        torch.empty(1 << 20, dtype=torch.uint8, device=dev).fill_(255)
    side.synchronize()
    for o in outs:
        assert torch.equal(o, want)
    q2, out = q.clone(), torch.empty_like(q)
    ws = ck.prefix_attention_workspace(q2, c.k_cache, c.prefix_len, c.max_len)
    run_prefix(c, q2, out=out, workspace=ws)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        run_prefix(c, q2, out=out, workspace=ws)
    q2.copy_(q.flip(0))
    c.seq_lens.copy_(torch.tensor([0, 2, 90, 200], dtype=torch.int32))  # lengths are the device's: a replay sees them
    graph.replay()
    torch.cuda.synchronize()
    replayed = out.clone()
    assert torch.equal(replayed, run_prefix(c, q2))
    poll_ok()
