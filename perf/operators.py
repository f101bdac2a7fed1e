"""The attention operators between a block's qkv projection and its output projection, as cases to measure.

Four operators: the norm and position rotation of query and key heads, the append of keys and values to a
paged cache, attention over that cache for a batch that shares a prefix, and cross attention to states of
another length.  Where ``own`` is false, ``run`` computes each in its plain form, elementary torch operations
in 32 bits rounded once at the end; where it is true it calls the package's entry points.  ``exact`` is the
definition in 64 bits.
"""
from __future__ import annotations

import math

import torch

own = False

BF16 = torch.bfloat16


# ---------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------

def _norm(name, T, Hq, Hk, D, rot, mode):
    return {"name": name, "op": "qk_norm_rope", "T": T, "Hq": Hq, "Hk": Hk, "D": D, "rot": rot, "mode": mode}


def _append(name, T, Hkv, D, rot, mode, page):
    return {"name": name, "op": "kv_append", "T": T, "Hkv": Hkv, "D": D, "rot": rot, "mode": mode, "page": page}


def _prefix(name, B, Lq, Hq, Hkv, D, page, prefix, suffix):
    return {"name": name, "op": "prefix_attention", "B": B, "Lq": Lq, "Hq": Hq, "Hkv": Hkv, "D": D,
            "page": page, "prefix": prefix, "suffix": suffix}


def _cross(name, B, Lq, Lk, Hq, Hkv, D):
    return {"name": name, "op": "cross_attention", "B": B, "Lq": Lq, "Lk": Lk, "Hq": Hq, "Hkv": Hkv, "D": D}


def listed():
    return [
        # one decode step of 16 sequences: launch latency
        _norm("norm_rope_decode", 16, 32, 8, 128, 128, "half"),
        # one block's 4096 image tokens, every head its own keys, pairs side by side
        _norm("norm_rope_block", 4096, 32, 32, 128, 128, "interleaved"),
        # a long ragged prefill, rotation of half of each head
        _norm("norm_rope_prefill", 30011, 40, 8, 128, 64, "half"),
        # one decode step of 64 sequences into small pages
        _append("append_decode", 64, 8, 128, 128, "half", 16),
        # a packed prefill of many prompts
        _append("append_prefill", 65519, 8, 128, 128, "half", 64),
        # a few sequences behind a short system prompt: latency
        _prefix("prefix_small", 4, 1, 32, 8, 128, 16, 1000, 130),
        # ordinary serving: a batch behind a long prompt, ragged answers
        _prefix("prefix_serving", 32, 1, 32, 8, 128, 16, 8192, 1024),
        # five draft tokens a sequence, an odd head group, 64-wide heads, pages that end inside a tile
        _prefix("prefix_draft", 7, 5, 24, 4, 64, 32, 4001, 777),
        # a large batch behind a document: the prefix is bound by arithmetic, the suffixes by memory
        _prefix("prefix_large", 128, 1, 64, 8, 128, 64, 32768, 4096),
        # an encoder-decoder's decode step
        _cross("cross_token", 16, 1, 1500, 16, 16, 64),
        # image tokens against a prompt's text states, ragged
        _cross("cross_block", 2, 4096, 333, 32, 32, 128),
        # long queries against long states, shared key heads
        _cross("cross_long", 2, 8192, 4093, 32, 8, 128),
    ]


def _log_int(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    case = _draw(rng)
    del case["name"]
    return case


def _draw(rng):
    op = rng.choice(["qk_norm_rope", "kv_append", "prefix_attention", "cross_attention"])
    if op == "qk_norm_rope":
        D = rng.choice([64, 96, 128, 256])
        Hk = rng.choice([1, 2, 4, 8, 32])
        Hq = Hk * rng.choice([1, 3, 4, 5]) if Hk < 32 else 32
        T = _log_int(rng, 1, 30011)
        T = min(T, 30011 * 48 * 128 // ((Hq + Hk) * D))
        return _norm("", T, Hq, Hk, D, rng.choice([D, D // 2]), rng.choice(["half", "interleaved"]))
    if op == "kv_append":
        D = rng.choice([64, 128])
        Hkv = rng.choice([1, 4, 5, 8])
        return _append("", _log_int(rng, 1, 65519), Hkv, D, rng.choice([0, D // 2, D]),
                       rng.choice(["half", "interleaved"]), rng.choice([16, 32, 64, 128]))
    if op == "prefix_attention":
        D = rng.choice([64, 128])
        Hkv = rng.choice([1, 2, 4, 8])
        G = rng.choice([1, 3, 4, 6, 8])
        B, Lq = _log_int(rng, 1, 128), rng.choice([1, 1, 2, 5])
        prefix, suffix = _log_int(rng, 1, 32768), _log_int(rng, 1, 4096)
        B = max(1, B // Lq)
        return _prefix("", B, Lq, Hkv * G, Hkv, D, rng.choice([16, 32, 64, 128]), prefix, suffix)
    D = rng.choice([64, 128])
    Hkv = rng.choice([1, 2, 8, 16])
    Hq = Hkv * rng.choice([1, 2, 3])
    Lq, Lk = _log_int(rng, 1, 8192), _log_int(rng, 1, 4093)
    B = _log_int(rng, 1, 16)
    while B * Lq * Lk * Hq > 8192 * (1024 + 4093) * 32:  # the largest listed one's pairs
        B = max(1, B // 2)
        if B == 1:
            Lq = max(1, Lq // 2)
    return _cross("", B, Lq, Lk, Hq, Hkv, D)


def _spread(n, top):
    """n lengths from 0 (one alone: top) to top, evenly spread."""
    if n == 1:
        return [top]
    return [int(round(top * i / (n - 1))) for i in range(n)]


def _cross_lens(case):
    """Lengths of the states of each sequence: from about a quarter to the whole."""
    B, Lk = case["B"], case["Lk"]
    low = (Lk + 3) // 4
    return [low + v for v in _spread(B, Lk - low)]


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------

def _randn(gen, *shape, std=1.0):
    t = torch.empty(shape, dtype=BF16, device="cuda")
    t.normal_(0.0, std, generator=gen)
    return t


def _table(max_pos, rot):
    """cos then sin of the usual angles, f32 [max_pos, rot]."""
    inv = 10000.0 ** (-torch.arange(0, rot, 2, dtype=torch.float64, device="cuda") / rot)
    ang = torch.arange(max_pos, dtype=torch.float64, device="cuda")[:, None] * inv[None, :]
    return torch.cat([ang.cos(), ang.sin()], 1).float()


def _inputs(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(int(seed) % (1 << 62))
    s = {"op": case["op"], "case": case}
    D = case["D"]
    if case["op"] == "qk_norm_rope":
        T, Hq, Hk = case["T"], case["Hq"], case["Hk"]
        qkv = _randn(gen, T, (Hq + 2 * Hk) * D, std=2.0)  # a packed projection: q and k are views of its rows
        s["q"] = qkv[:, :Hq * D].view(T, Hq, D)
        s["k"] = qkv[:, Hq * D:(Hq + Hk) * D].view(T, Hk, D)
        s["wq"] = (1.0 + 0.2 * torch.randn(D, generator=gen, device="cuda")).to(BF16)
        s["wk"] = (1.0 + 0.2 * torch.randn(D, generator=gen, device="cuda")).to(BF16)
        s["max_pos"] = max(4096, T)
        s["table"] = _table(s["max_pos"], case["rot"])
        s["pos"] = torch.randint(0, s["max_pos"], (T,), generator=gen, device="cuda", dtype=torch.int32)
    elif case["op"] == "kv_append":
        T, H, page = case["T"], case["Hkv"], case["page"]
        kv = _randn(gen, T, 2 * H * D, std=2.0)
        s["k"] = kv[:, :H * D].view(T, H, D)
        s["v"] = kv[:, H * D:].view(T, H, D)
        s["wk"] = (1.0 + 0.2 * torch.randn(D, generator=gen, device="cuda")).to(BF16)
        pages = (T + page - 1) // page + 1
        s["kc"] = torch.zeros(pages, H, page, D, dtype=BF16, device="cuda")
        s["vc"] = torch.zeros(pages, H, page, D, dtype=BF16, device="cuda")
        # whole pages in any order, tokens in order within a page; every 17th token is padding
        order = torch.randperm(pages, generator=gen, device="cuda")
        t = torch.arange(T, device="cuda")
        slots = order[t // page] * page + t % page
        s["slots"] = torch.where(t % 17 == 16, torch.full_like(slots, -1), slots)
        s["max_pos"] = max(4096, T)
        s["table"] = _table(s["max_pos"], case["rot"]) if case["rot"] else None
        s["pos"] = torch.randint(0, s["max_pos"], (T,), generator=gen, device="cuda", dtype=torch.int32)
    elif case["op"] == "prefix_attention":
        B, Lq, Hq, H, page = case["B"], case["Lq"], case["Hq"], case["Hkv"], case["page"]
        lens = _spread(B, case["suffix"])
        perm = torch.randperm(B, generator=gen, device="cuda").tolist()
        lens = [lens[i] for i in perm]
        per = [(n + page - 1) // page for n in lens]
        npre = (case["prefix"] + page - 1) // page
        pages = npre + sum(per) + 1
        order = torch.randperm(pages, generator=gen, device="cuda").to(torch.int32)
        s["prefix_pages"] = order[:npre].contiguous()
        width = max(1, (case["suffix"] + page - 1) // page)
        table = torch.zeros(B, width, dtype=torch.int32)
        host, at = order.cpu(), npre
        for b in range(B):
            table[b, :per[b]] = host[at:at + per[b]]
            at += per[b]
        s["block_table"] = table.cuda()
        s["lens"], s["seq_lens"] = lens, torch.tensor(lens, dtype=torch.int32, device="cuda")
        s["kc"] = _randn(gen, pages, H, page, D)
        s["vc"] = _randn(gen, pages, H, page, D)
        s["q"] = _randn(gen, B, Lq, Hq, D, std=1.5)
    else:
        B, Lq, Lk, Hq, H = case["B"], case["Lq"], case["Lk"], case["Hq"], case["Hkv"]
        lens = _cross_lens(case)
        perm = torch.randperm(B, generator=gen, device="cuda").tolist()
        s["lens"] = [lens[i] for i in perm]
        s["kv_lens"] = torch.tensor(s["lens"], dtype=torch.int32, device="cuda")
        s["q"] = _randn(gen, B, Lq, Hq, D, std=1.5)
        kv = _randn(gen, B, Lk, 2 * H * D)  # one packed projection of the states
        s["k"] = kv[:, :, :H * D].view(B, Lk, H, D)
        s["v"] = kv[:, :, H * D:].view(B, Lk, H, D)
    return s


def prepare(case, seed):
    s = _inputs(case, seed)
    if own:
        import swiglu_mlp_group_gb300 as ck
        if case["op"] == "prefix_attention":
            s["ws"] = ck.prefix_attention_workspace(s["q"], s["kc"], case["prefix"], case["suffix"])
        elif case["op"] == "cross_attention":
            s["ws"] = ck.cross_attention_workspace(s["q"], s["k"])
    return s


# ---------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------

def run(state):
    return (_own if own else _plain)(state)


def _own(s):
    import swiglu_mlp_group_gb300 as ck
    c = s["case"]
    if s["op"] == "qk_norm_rope":
        return ck.qk_norm_rope(s["q"], s["k"], s["table"], s["pos"], wq=s["wq"], wk=s["wk"], eps=1e-6,
                               mode=c["mode"])
    if s["op"] == "kv_append":
        ck.kv_append(s["k"], s["v"], s["kc"], s["vc"], s["slots"], cos_sin=s["table"], positions=s["pos"],
                     wk=s["wk"], eps=1e-6, mode=c["mode"])
        return s["kc"], s["vc"]
    if s["op"] == "prefix_attention":
        return ck.prefix_attention(s["q"], s["kc"], s["vc"], s["prefix_pages"], c["prefix"],
                                   s["block_table"], s["seq_lens"], c["suffix"], workspace=s["ws"])
    return ck.cross_attention(s["q"], s["k"], s["v"], kv_lens=s["kv_lens"], workspace=s["ws"])


def _plain_norm_rope(x, w, table, pos, mode):
    """x [T, H, D] -> f32 [T, H, D]."""
    y = x.float()
    y = y * torch.rsqrt((y * y).mean(-1, keepdim=True) + 1e-6) * w.float()
    if table is None:
        return y
    rot = table.shape[1]
    cs = table[pos.long()]
    cos, sin = cs[:, None, :rot // 2], cs[:, None, rot // 2:]
    out = y.clone()
    if mode == "half":
        a, b = y[..., :rot // 2], y[..., rot // 2:rot]
        out[..., :rot // 2] = a * cos - b * sin
        out[..., rot // 2:rot] = b * cos + a * sin
    else:
        a, b = y[..., 0:rot:2], y[..., 1:rot:2]
        out[..., 0:rot:2] = a * cos - b * sin
        out[..., 1:rot:2] = b * cos + a * sin
    return out


def _plain_attend(q, k, v, seen):
    """q f32 [H, R, D], k and v f32 [H, n, D], seen: truth values [R, n] or None -> (max, sum, unscaled output)."""
    x = q @ k.transpose(1, 2)
    if seen is not None:
        x = x.masked_fill(~seen, -math.inf)
    m = x.amax(-1, keepdim=True) if k.shape[1] else torch.full_like(q[..., :1], -math.inf)
    p = torch.exp(x - torch.where(m == -math.inf, torch.zeros_like(m), m))
    return m, p.sum(-1, keepdim=True), p @ v


def _plain_heads(q, k, v):
    """_plain_attend of all keys, as many heads at once as 2 GB of scores hold."""
    n = max(1, (1 << 29) // max(1, q.shape[1] * k.shape[1]))
    parts = [_plain_attend(q[h:h + n], k[h:h + n], v[h:h + n], None) for h in range(0, q.shape[0], n)]
    return [torch.cat(t) for t in zip(*parts)]


def _plain_pages(cache, pages, n):
    """f32 [Hkv, n, D] of the first n tokens of the given pages."""
    t = cache[pages.long()].float()
    return t.permute(1, 0, 2, 3).reshape(cache.shape[1], -1, cache.shape[3])[:, :n]


def _plain(s):
    c = s["case"]
    if s["op"] == "qk_norm_rope":
        return tuple(_plain_norm_rope(s[x], s["w" + x], s["table"], s["pos"], c["mode"]).to(BF16) for x in "qk")
    if s["op"] == "kv_append":
        k = _plain_norm_rope(s["k"], s["wk"], s["table"], s["pos"], c["mode"]).to(BF16)
        keep = torch.nonzero(s["slots"] >= 0)[:, 0]
        at = s["slots"][keep]
        s["kc"][at // c["page"], :, at % c["page"]] = k[keep]
        s["vc"][at // c["page"], :, at % c["page"]] = s["v"][keep]
        return s["kc"], s["vc"]
    q = s["q"]
    B, Lq, Hq, D = q.shape
    H = c["Hkv"]
    G = Hq // H
    out = torch.empty(B, Lq, Hq, D, dtype=BF16, device=q.device)
    # rows of one sequence by key head: [B, H, Lq * G, D]
    rows = q.float().mul(1.0 / math.sqrt(D)).view(B, Lq, H, G, D).permute(0, 2, 1, 3, 4).reshape(B, H, Lq * G, D)
    if s["op"] == "prefix_attention":
        kp, vp = (_plain_pages(s[x], s["prefix_pages"], c["prefix"]) for x in ("kc", "vc"))
        one = rows.permute(1, 0, 2, 3).reshape(H, B * Lq * G, D)
        shared = [t.view(H, B, Lq * G, -1) for t in _plain_heads(one, kp, vp)]
        token = torch.arange(Lq * G, device=q.device) // G
    for b in range(B):
        n = s["lens"][b]
        if s["op"] == "prefix_attention":
            pages = s["block_table"][b, :(n + c["page"] - 1) // c["page"]]
            k, v = (_plain_pages(s[x], pages, n) for x in ("kc", "vc"))
            seen = torch.arange(n, device=q.device)[None, :] <= (n - Lq + token)[:, None]
            m, l, o = _plain_attend(rows[b], k, v, seen)
            pm, pl, po = (t[:, b] for t in shared)
            top = torch.maximum(m, pm)
            f, pf = torch.exp(m - top), torch.exp(pm - top)
            o, l = o * f + po * pf, l * f + pl * pf
            o = o / l
        else:
            k, v = (s[x][b, :n].float().transpose(0, 1) for x in "kv")
            _, l, o = _plain_heads(rows[b], k, v)
            o = o / l
        out[b] = o.view(H, Lq, G, D).transpose(0, 1).reshape(Lq, Hq, D)
    return out


# ---------------------------------------------------------------------------
# what a pass cannot do without
# ---------------------------------------------------------------------------

def work(case):
    D = case["D"]
    if case["op"] == "qk_norm_rope":
        n = case["T"] * (case["Hq"] + case["Hk"]) * D
        return {"bytes": 4 * n + 4 * case["T"] * (1 + case["rot"]), "flops": 10 * n}
    if case["op"] == "kv_append":
        n = case["T"] * case["Hkv"] * D
        kept = case["T"] - case["T"] // 17
        return {"bytes": (4 * n + 4 * kept * case["Hkv"] * D) + case["T"] * (12 + 4 * case["rot"]), "flops": 10 * n}
    if case["op"] == "prefix_attention":
        B, Lq = case["B"], case["Lq"]
        lens = _spread(B, case["suffix"])
        pairs = B * Lq * case["prefix"] + sum(max(0, n - Lq + i + 1) for n in lens for i in range(Lq))
        return {"bytes": 4 * B * Lq * case["Hq"] * D + 4 * case["Hkv"] * D * (case["prefix"] + sum(lens)),
                "flops": 4 * case["Hq"] * D * pairs}
    keys = sum(_cross_lens(case))
    return {"bytes": 4 * case["B"] * case["Lq"] * case["Hq"] * D + 4 * case["Hkv"] * D * keys,
            "flops": 4 * case["Hq"] * D * case["Lq"] * keys}


# ---------------------------------------------------------------------------
# the definitions in 64 bits
# ---------------------------------------------------------------------------

def _exact_head(x, w, table, pos, mode):
    """Norm and rotation by complex numbers: x [T, H, D] -> f64."""
    x = x.double()
    x = w.double() * x / torch.sqrt(torch.einsum("thd,thd->th", x, x)[..., None] / x.shape[-1] + 1e-6)
    if table is None:
        return x
    r = table.shape[1]
    cs = table.double().index_select(0, pos.long())
    turn = torch.complex(cs[:, :r // 2].contiguous(), cs[:, r // 2:].contiguous())[:, None]
    pair = x[..., :r].unflatten(-1, (2, r // 2)).transpose(-1, -2) if mode == "half" else x[..., :r].unflatten(-1, (r // 2, 2))
    z = torch.view_as_real(torch.view_as_complex(pair.contiguous()) * turn)
    z = z.transpose(-1, -2) if mode == "half" else z
    return torch.cat([z.flatten(-2), x[..., r:]], -1)


def _exact_softmax(q, k, v, last):
    """q [R, D], k and v [n, D] in f64; row r sees keys 0 .. last[r] - 1."""
    out = torch.zeros(q.shape[0], v.shape[1], dtype=torch.float64, device=q.device)
    step = max(1, (1 << 28) // max(1, k.shape[0]))
    at = torch.arange(k.shape[0], device=q.device)
    for r in range(0, q.shape[0], step):
        z = torch.einsum("rd,nd->rn", q[r:r + step], k) / math.sqrt(q.shape[1])
        z.masked_fill_(at >= last[r:r + step, None], -math.inf)
        out[r:r + step] = torch.softmax(z, -1).nan_to_num(0.0) @ v
    return out


def exact(case, seed):
    s = _inputs(case, seed)
    if case["op"] == "qk_norm_rope":
        return tuple(_exact_head(s[x], s["w" + x], s["table"], s["pos"], case["mode"]) for x in "qk")
    if case["op"] == "kv_append":
        keys = _exact_head(s["k"], s["wk"], s["table"], s["pos"], case["mode"])
        done = []
        for cache, new in ((s["kc"], keys), (s["vc"], s["v"].double())):
            flat = cache.double().transpose(1, 2).reshape(-1, case["Hkv"], case["D"])  # by slot
            real = s["slots"] >= 0
            flat.index_copy_(0, s["slots"][real], new[real])
            done.append(flat.view(-1, case["page"], case["Hkv"], case["D"]).transpose(1, 2).contiguous())
        return tuple(done)
    B, Lq, Hq, D = s["q"].shape
    H = case["Hkv"]
    G = Hq // H
    if 4.0 * D * Hq * B * Lq * (case.get("prefix", 0) + case.get("suffix", 0) + case.get("Lk", 0)) > 4e12:
        return None
    out = torch.empty(B, Lq, Hq, D, dtype=torch.float64, device="cuda")
    token = torch.arange(Lq, device="cuda").repeat_interleave(G)
    for h in range(H):
        if case["op"] == "prefix_attention":
            front = [s[x][s["prefix_pages"].long(), h].double().flatten(0, 1)[:case["prefix"]] for x in ("kc", "vc")]
        for b in range(B):
            n = s["lens"][b]
            q = s["q"][b, :, h * G:(h + 1) * G].double().reshape(Lq * G, D)
            if case["op"] == "prefix_attention":
                own_pages = s["block_table"][b].long()
                k, v = (torch.cat([f, s[x][own_pages, h].double().flatten(0, 1)[:n]])
                        for f, x in zip(front, ("kc", "vc")))
                last = case["prefix"] + (n - Lq + token + 1).clamp(min=0)
            else:
                k, v = s["k"][b, :n, h].double(), s["v"][b, :n, h].double()
                last = torch.full((Lq * G,), n, device="cuda")
            out[b, :, h * G:(h + 1) * G] = _exact_softmax(q, k, v, last).view(Lq, G, D)
    return out
