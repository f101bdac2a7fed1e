"""Microscaled 4-bit linears and the norms between a block's parts, as cases to measure.

Four operators: the norm of a residual stream with the sum, gate and modulation ahead of it; the same with its
result quantized to 4-bit floats and multiplied by a 4-bit weight; the linear on bf16 activations (quantized on
the way) and 4-bit weights, from one token to long prompts; and the SwiGLU MLP of two such linears.  Formats:
``mx`` (32 codes share a power of two) and ``nv`` (16 codes share an E4M3 scale, and a tensor one f32 scale).
Where ``own`` is false, ``run`` computes each in its plain form, elementary torch operations in 32 bits rounded
once at the end; where it is true it calls the package's entry points.  ``exact`` is the definition in 64 bits.
"""
from __future__ import annotations

import math

import torch

own = False

BF16 = torch.bfloat16
BLOCK = {"mx": 32, "nv": 16}
E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)
EPS = 1e-6


# ---------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------

def _norm(name, T, H, kind, post, mod, per_group):
    """mod: "none", "gate" (one row for all tokens) or "full" (gate, scale and shift of every per_group tokens)."""
    return {"name": name, "op": "block_norm", "T": T, "H": H, "kind": kind, "post": post, "mod": mod,
            "per_group": per_group}


def _norm_linear(name, T, H, N, fmt, kind, post, mod, per_group):
    return {"name": name, "op": "norm_linear", "T": T, "H": H, "N": N, "fmt": fmt, "kind": kind, "post": post,
            "mod": mod, "per_group": per_group}


def _linear(name, M, K, N, fmt, bias, residual):
    return {"name": name, "op": "linear", "M": M, "K": K, "N": N, "fmt": fmt, "bias": bias, "residual": residual}


def _mlp(name, M, H, I, fmt, residual):
    return {"name": name, "op": "swiglu_mlp", "M": M, "H": H, "I": I, "fmt": fmt, "residual": residual}


def listed():
    return [
        # a decode step of 16 sequences, residual sum and norm: launch latency
        _norm("norm_decode", 16, 4096, "rms", False, "none", 0),
        # layer norm with bias behind a per-channel gate, an odd width and an odd number of tokens
        _norm("norm_odd", 777, 1160, "layer", False, "gate", 0),
        # a long ragged prefill with norms on both sides of the branch
        _norm("norm_prefill", 30011, 5120, "rms", True, "none", 0),
        # a decode step's norm in front of its qkv projection
        _norm_linear("norm_linear_decode", 8, 4096, 6144, "nv", "rms", False, "none", 0),
        # an image block: two samples' gate, scale and shift, in front of its gate|up-sized projection
        _norm_linear("norm_linear_block", 4096, 4096, 12288, "mx", "layer", False, "full", 2048),
        # one token against a wide weight: the weight's bytes
        _linear("linear_token", 1, 4096, 12288, "nv", False, False),
        # a few draft tokens, the down projection, with bias and skip connection
        _linear("linear_few", 13, 12288, 4096, "mx", True, True),
        # ragged sizes: nothing is a multiple of a tile
        _linear("linear_ragged", 1000, 2080, 1544, "nv", True, False),
        # one block's tokens
        _linear("linear_block", 4096, 4096, 4096, "mx", False, False),
        # a long prefill: the tensor cores' rate
        _linear("linear_prefill", 16384, 4096, 12288, "nv", False, False),
        # a decode step's MLP
        _mlp("mlp_few", 5, 4096, 12288, "nv", True),
        # an image block's MLP
        _mlp("mlp_block", 4096, 4096, 12288, "mx", True),
    ]


def _log_int(rng, lo, hi, of=1):
    v = math.exp(rng.uniform(math.log(lo), math.log(hi)))
    return min(hi // of, max(-(-lo // of), int(round(v / of)))) * of


def draw(rng):
    case = _draw(rng)
    del case["name"]
    return case


def _draw(rng):
    op = rng.choice(["block_norm", "norm_linear", "linear", "swiglu_mlp"])
    kind, post, fmt = rng.choice(["rms", "layer"]), rng.choice([True, False]), rng.choice(["mx", "nv"])
    mod = rng.choice(["none", "gate", "full"])
    if op == "block_norm":
        H = _log_int(rng, 64, 8192, 8)
        T = min(_log_int(rng, 1, 30011), 30011 * 5120 // H)
        return _norm("", T, H, kind, post, mod, _log_int(rng, 1, T) if mod == "full" else 0)
    cap = 16384 * 4096 * 12288  # the largest listed one's products
    M = _log_int(rng, 1, 16384)
    if op == "swiglu_mlp":
        H, I = _log_int(rng, 128, 8192, 32), _log_int(rng, 128, 12288, 32)
        return _mlp("", max(1, min(M, cap // (3 * H * I))), H, I, fmt, rng.choice([True, False]))
    K, N = _log_int(rng, 96, 12288, 32), _log_int(rng, 64, 24576, 8)
    if op == "linear":
        M = max(1, min(M, cap // (K * N)))
        return _linear("", M, K, N, fmt, rng.choice([True, False]), rng.choice([True, False]))
    K = min(K, 8192)
    M = max(1, min(M, cap // (K * N)))
    return _norm_linear("", M, K, N, fmt, kind, post, mod, _log_int(rng, 1, M) if mod == "full" else 0)


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------

def _gen(seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(int(seed) % (1 << 62))
    return gen


def _randn(gen, *shape, std=1.0, mean=0.0):
    t = torch.empty(shape, dtype=BF16, device="cuda")
    return t.normal_(mean, std, generator=gen)


def _activation(gen, M, K):
    """Normal values, every 97th channel ten times as large."""
    x = _randn(gen, M, K)
    x[:, 11 % K::97] *= 10
    return x


def _weight(s, name, gen, N, K, fmt):
    """A 4-bit weight as a checkpoint holds it: codes two to a byte (the first in the low half), block scales by row."""
    w = _randn(gen, N, K, std=1.0 / math.sqrt(K)).float()
    t = float(w.abs().max()) / 2688.0 if fmt == "nv" else 1.0
    codes, scales, _ = _plain_quantize(w, fmt, t)
    s[name] = (codes[:, 0::2] | codes[:, 1::2] << 4).contiguous()
    s[name + "_scales"], s[name + "_t"] = scales, t


def _inputs(case, seed):
    gen = _gen(seed)
    s = {"op": case["op"], "case": case}
    fmt = case.get("fmt")
    # scales of the activations, as a calibration leaves them: some f32 number (of a short fraction, many values would
    # lie on the border between two codes)
    s["x_t"], s["a_t"] = (0.01674109, 0.004463737) if fmt == "nv" else (1.0, 1.0)
    if case["op"] in ("block_norm", "norm_linear"):
        T, H = case["T"], case["H"]
        s["x"], s["branch"] = _activation(gen, T, H), _randn(gen, T, H, std=0.7, mean=0.1)
        s["weight"] = _randn(gen, H, std=0.2, mean=1.0)
        s["bias"] = _randn(gen, H, std=0.1) if case["kind"] == "layer" else None
        s["post_weight"] = _randn(gen, H, std=0.2, mean=1.0) if case["post"] else None
        s["factor"] = 0.75 if case["post"] else 1.0  # of the branch, in the sum
        s["per_group"] = case["per_group"]
        s["gate"] = s["scale"] = s["shift"] = None
        if case["mod"] == "gate":
            s["gate"] = _randn(gen, 1, H, std=0.3)
        elif case["mod"] == "full":  # rows of one modulation projection
            rows = -(-T // case["per_group"])
            m = _randn(gen, rows, 3 * H, std=0.3)
            s["gate"], s["scale"], s["shift"] = m[:, :H], m[:, H:2 * H], m[:, 2 * H:]
        if case["op"] == "norm_linear":
            s["x_t"] = 0.003732391 if fmt == "nv" else 1.0
            _weight(s, "w", gen, case["N"], H, fmt)
    elif case["op"] == "linear":
        M, K, N = case["M"], case["K"], case["N"]
        s["x"] = _activation(gen, M, K)
        _weight(s, "w", gen, N, K, fmt)
        s["bias"] = _randn(gen, N, std=0.1) if case["bias"] else None
        s["residual"] = _randn(gen, M, N) if case["residual"] else None
    else:
        M, H, I = case["M"], case["H"], case["I"]
        s["x"] = _activation(gen, M, H)
        _weight(s, "gate_up", gen, 2 * I, H, fmt)
        _weight(s, "down", gen, H, I, fmt)
        s["residual"] = _randn(gen, M, H) if case["residual"] else None
    return s


def prepare(case, seed):
    s = _inputs(case, seed)
    if own:
        import swiglu_mlp_group_gb300 as ck
        for name in ("w", "gate_up", "down"):  # the scales in the order that the tensor cores read them, once
            if name in s:
                s[name + "_tiled"] = ck.fp4_tile_scales(s[name + "_scales"], case["fmt"])
        if case["op"] == "linear":
            s["ws"] = ck.fp4_linear_workspace(case["M"], case["K"], case["fmt"])
        elif case["op"] == "swiglu_mlp":
            s["ws"] = ck.fp4_swiglu_mlp_workspace(case["M"], case["H"], case["I"], case["fmt"])
    return s


# ---------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------

def run(state):
    return (_own if own else _plain)(state)


def _own(s):
    import swiglu_mlp_group_gb300 as ck
    c = s["case"]
    if s["op"] in ("block_norm", "norm_linear"):
        args = dict(post_weight=s["post_weight"], gate=s["gate"], branch_factor=s["factor"], norm=c["kind"],
                    weight=s["weight"], bias=s["bias"], scale=s["scale"], shift=s["shift"],
                    tokens_per_group=s["per_group"], eps=EPS)
        if s["op"] == "block_norm":
            return ck.block_norm(s["x"], s["branch"], **args)
        h, codes, scales = ck.block_norm_fp4(s["x"], s["branch"], fmt=c["fmt"], n_scale=s["x_t"], **args)
        return h, ck.fp4_gemm(codes, scales, s["w"], s["w_tiled"], c["fmt"], alpha=s["x_t"] * s["w_t"])
    if s["op"] == "linear":
        return ck.fp4_linear(s["x"], s["w"], s["w_tiled"], c["fmt"], x_scale=s["x_t"], w_scale=s["w_t"],
                             bias=s["bias"], residual=s["residual"], workspace=s["ws"])
    return ck.fp4_swiglu_mlp(s["x"], s["gate_up"], s["gate_up_tiled"], s["down"], s["down_tiled"], c["fmt"],
                             x_scale=s["x_t"], gate_up_scale=s["gate_up_t"], act_scale=s["a_t"],
                             down_scale=s["down_t"], residual=s["residual"], workspace=s["ws"])


def _plain_quantize(x, fmt, t):
    """f32 [M, K] -> (codes uint8 [M, K], block scales uint8 [M, K / block], values f32 [M, K])."""
    M, K = x.shape
    b = x.view(M, K // BLOCK[fmt], BLOCK[fmt])
    amax = b.abs().amax(-1)
    if fmt == "mx":
        # the exponent of the largest value, less that of the largest code
        exponent = (amax.view(torch.int32) >> 23).sub(2).clamp(min=0)
        scales = exponent.to(torch.uint8)
        d = torch.exp2(exponent.float() - 127.0)
    else:
        s8 = (amax / (6.0 * torch.tensor(t, dtype=torch.float32, device=x.device))).clamp(max=448.0).to(torch.float8_e4m3fn)
        scales = s8.view(torch.uint8)
        d = s8.float() * torch.tensor(t, dtype=torch.float32, device=x.device)
    q = b / torch.where(d == 0, torch.full_like(d, math.inf), d).unsqueeze(-1)
    a = q.abs()
    # the border between two codes belongs to the even one
    code = ((a > 0.25).byte() + (a >= 0.75) + (a > 1.25) + (a >= 1.75) + (a > 2.5) + (a >= 3.5) + (a > 5.0)).view(M, K)
    code = code | (q < 0).view(M, K).byte() << 3
    return code, scales, _plain_values(code, scales, fmt, t)


def _plain_values(code, scales, fmt, t):
    """The values that codes and scales stand for, f32."""
    M, K = code.shape
    table = torch.tensor(E2M1 + tuple(-v for v in E2M1), dtype=torch.float32, device=code.device)
    d = torch.exp2(scales.float() - 127.0) if fmt == "mx" else scales.view(torch.float8_e4m3fn).float() * t
    return (table[code.int()].view(M, K // BLOCK[fmt], BLOCK[fmt]) * d.unsqueeze(-1)).view(M, K)


def _plain_weight(s, name, fmt):
    w = s[name]
    return _plain_values(torch.stack([w & 15, w >> 4], -1).view(w.shape[0], -1), s[name + "_scales"], fmt, s[name + "_t"])


def _plain_norm(s):
    """(h, n) in f32."""
    c = s["case"]
    x, b = s["x"].float(), s["branch"].float()
    rows = torch.arange(c["T"], device=x.device) // (c["per_group"] or c["T"])
    if s["post_weight"] is not None:
        b = b * torch.rsqrt((b * b).mean(-1, keepdim=True) + EPS) * s["post_weight"].float()
    if s["gate"] is not None:
        b = b * s["gate"].float()[rows]
    h = x + s["factor"] * b
    n = h
    if c["kind"] == "layer":
        n = n - n.mean(-1, keepdim=True)
    n = n * torch.rsqrt((n * n).mean(-1, keepdim=True) + EPS) * s["weight"].float()
    if s["bias"] is not None:
        n = n + s["bias"].float()
    if s["scale"] is not None:
        n = n * (1.0 + s["scale"].float()[rows]) + s["shift"].float()[rows]
    return h, n


def _plain(s):
    c = s["case"]
    fmt = c.get("fmt")
    if s["op"] in ("block_norm", "norm_linear"):
        h, n = _plain_norm(s)
        if s["op"] == "norm_linear":
            n = _plain_quantize(n, fmt, s["x_t"])[2] @ _plain_weight(s, "w", fmt).t()
        return h.to(BF16), n.to(BF16)
    x = _plain_quantize(s["x"].float(), fmt, s["x_t"])[2]
    if s["op"] == "linear":
        y = x @ _plain_weight(s, "w", fmt).t()
        if s["bias"] is not None:
            y = y + s["bias"].float()
    else:
        h = (x @ _plain_weight(s, "gate_up", fmt).t()).to(BF16).float()  # h is bf16 between the two linears
        gate, up = h[:, :c["I"]], h[:, c["I"]:]
        a = gate / (1.0 + torch.exp(-gate)) * up
        y = _plain_quantize(a.contiguous(), fmt, s["a_t"])[2] @ _plain_weight(s, "down", fmt).t()
    if s["residual"] is not None:
        y = y + s["residual"].float()
    return y.to(BF16)


# ---------------------------------------------------------------------------
# what a pass cannot do without
# ---------------------------------------------------------------------------

def _weight_bytes(N, K, fmt):
    return N * K // 2 + N * K // BLOCK[fmt]


def work(case):
    if case["op"] in ("block_norm", "norm_linear"):
        T, H = case["T"], case["H"]
        rows = 0 if case["mod"] != "full" else -(-T // case["per_group"])
        vectors = 1 + (case["kind"] == "layer") + case["post"] + (case["mod"] == "gate") + 3 * rows
        w = {"bytes": 6 * T * H + 2 * H * vectors, "flops": 12 * T * H}
        if case["op"] == "block_norm":
            w["bytes"] += 2 * T * H
        else:
            w["bytes"] += _weight_bytes(case["N"], H, case["fmt"]) + 2 * T * case["N"]
            w["flops"] += 2 * T * H * case["N"]
        return w
    M = case["M"]
    if case["op"] == "linear":
        K, N = case["K"], case["N"]
        return {"bytes": 2 * M * K + _weight_bytes(N, K, case["fmt"]) + 2 * M * N * (1 + case["residual"])
                + 2 * N * case["bias"], "flops": 2 * M * N * K}
    H, I = case["H"], case["I"]
    return {"bytes": 2 * M * H * (2 + case["residual"]) + _weight_bytes(2 * I, H, case["fmt"])
            + _weight_bytes(H, I, case["fmt"]), "flops": 6 * M * H * I}


# ---------------------------------------------------------------------------
# the definitions in 64 bits
# ---------------------------------------------------------------------------

def _exact_quantize(x, fmt, t):
    """f64 [M, K] -> the values that its codes and scales stand for, f64: each number rounded, half to even, to the
    step of its binade."""
    shape = x.shape
    x = x.reshape(-1, BLOCK[fmt])
    top = x.abs().max(dim=1, keepdim=True).values
    if fmt == "mx":
        d = torch.ldexp(torch.ones_like(top), (torch.frexp(top).exponent - 3).clamp(min=-127))
    else:
        t = float(torch.tensor(t, dtype=torch.float32))
        s = top / 6.0 / t
        step = torch.ldexp(torch.ones_like(s), (torch.frexp(s).exponent - 4).clamp(min=-9))
        d = (torch.round(s / step) * step).clamp(max=448.0) * t
    q = torch.where(d > 0, x / d, torch.zeros_like(x))
    step = torch.ldexp(torch.ones_like(q), torch.frexp(q).exponent.clamp(min=1) - 2)
    return ((torch.round(q / step) * step).clamp(-6.0, 6.0) * d).reshape(shape)


def _exact_weight(s, name, fmt):
    """Codes by their bits: value = (-1)^sign * (mantissa and hidden bit) / 2 * 2^max(exponent - 1, 0)."""
    w = s[name].to(torch.int64)
    code = torch.stack([w % 16, w // 16], 2).flatten(1)
    e, m = (code // 2) % 4, code % 2
    v = torch.ldexp((m + 2 * (e > 0)).double() / 2, (e - 1).clamp(min=0)) * (1 - 2 * (code // 8)).double()
    b = s[name + "_scales"].to(torch.int64)
    if fmt == "mx":
        d = torch.ldexp(torch.ones_like(b, dtype=torch.float64), b - 127)
    else:
        d = torch.where(b >= 8, torch.ldexp((b % 8 + 8).double(), b // 8 - 10), torch.ldexp((b % 8).double(), -9 + 0 * b))
        d = d * s[name + "_t"]
    return v * d.repeat_interleave(BLOCK[fmt], dim=1)


def _exact_norm(s):
    c = s["case"]
    per = c["per_group"] or c["T"]
    def spread(v):  # [groups, H] -> [T, H]
        return v.double().repeat_interleave(per, dim=0)[:c["T"]]
    b = s["branch"].double()
    if s["post_weight"] is not None:
        b = s["post_weight"].double() * b / (torch.einsum("th,th->t", b, b) / c["H"] + EPS).sqrt()[:, None]
    if s["gate"] is not None:
        b = spread(s["gate"]) * b
    h = torch.add(s["x"].double(), b, alpha=s["factor"])
    mean = h.mean(1, keepdim=True) if c["kind"] == "layer" else 0.0
    n = (h - mean) / ((h - mean).pow(2).mean(1, keepdim=True) + EPS).sqrt() * s["weight"].double()
    if s["bias"] is not None:
        n += s["bias"].double()
    if s["scale"] is not None:
        n = torch.addcmul(n, n, spread(s["scale"])) + spread(s["shift"])
    return h, n


def exact(case, seed):
    s = _inputs(case, seed)
    fmt = case.get("fmt")
    if case["op"] in ("block_norm", "norm_linear"):
        h, n = _exact_norm(s)
        if case["op"] == "block_norm":
            return h, n
        return h, torch.einsum("tk,nk->tn", _exact_quantize(n, fmt, s["x_t"]), _exact_weight(s, "w", fmt))
    x = _exact_quantize(s["x"].double(), fmt, s["x_t"])
    if case["op"] == "linear":
        y = torch.einsum("mk,nk->mn", x, _exact_weight(s, "w", fmt))
        if s["bias"] is not None:
            y += s["bias"].double()
    else:
        h = torch.einsum("mk,nk->mn", x, _exact_weight(s, "gate_up", fmt)).to(BF16).double()
        gate, up = h.chunk(2, dim=1)
        y = torch.einsum("mk,nk->mn", _exact_quantize(gate * torch.sigmoid(gate) * up, fmt, s["a_t"]),
                         _exact_weight(s, "down", fmt))
    if s["residual"] is not None:
        y += s["residual"].double()
    return y
