"""What is measured of the MXFP4 and MoE-gradient operators: the cases, their inputs, the operators in
plain torch operations and in 64 bits, and the calls that a user makes.

Operators (names and arguments as in group_gemm_amd):

* ``mxfp4_quantize(x)``, ``mxfp4_quantize_weights(w)``, ``mxfp4_dequantize(codes, scale)``: rows [rows, k] or
  expert weights [g, k, n] to 4-bit e2m1 codes with one power-of-two scale per 32 elements along k, and back.
* ``ragged_dot_m_mxfp4(lhs, rhs, group_sizes, lhs_scale, rhs_scale)``: the MoE product over such operands.
* ``moe_permute_grad`` and ``moe_unpermute_grad``: the gradients of the sort by expert and of the weighted way back.

Layouts: codes are two elements a byte along k, the even element in the low half; weights are [g, n, k/2].
Scales are in panels of 256 elements along k: [ceil(k/256), rows, 8] or [g, ceil(k/256), n, 8], one byte
(value 2^(byte - 127)) per 32 elements, zero past k.
"""
import math

import numpy as np
import torch

own = False
DEV = "cuda"
DT = {"bf16": torch.bfloat16, "f32": torch.float32}
FP4 = torch.float4_e2m1fn_x2


def listed():
    return [
        # a few decoding tokens' activations, a width that is no multiple of a panel: latency
        {"name": "quantize_tokens_small", "op": "quantize", "rows": 24, "k": 2880, "dtype": "f32"},
        # the activations of 4096 prompt tokens before they are sorted by expert
        {"name": "quantize_tokens", "op": "quantize", "rows": 4096, "k": 7168, "dtype": "bf16"},
        # eight experts' up-projections, quantised once when a model is loaded
        {"name": "quantize_weights", "op": "weights", "g": 8, "k": 4096, "n": 14336, "dtype": "bf16"},
        # one token at its two experts of eight: the weights of two experts are read once
        {"name": "product_one_token", "op": "product", "tokens": 1, "top_k": 2, "tail": 0, "k": 4096, "n": 14336, "g": 8, "skew": 0.0, "out": "bf16"},
        # 64 decoding tokens at four of 128 experts: one to a few rows each, many experts
        {"name": "product_decode", "op": "product", "tokens": 64, "top_k": 4, "tail": 0, "k": 2880, "n": 5760, "g": 128, "skew": 0.0, "out": "bf16"},
        # a small ragged batch with rows past the last group, n without any alignment, 32-bit output
        {"name": "product_odd", "op": "product", "tokens": 375, "top_k": 4, "tail": 13, "k": 2880, "n": 1447, "g": 32, "skew": 0.0, "out": "f32"},
        # prompt processing, eight experts with about 1000 rows each
        {"name": "product_prefill", "op": "product", "tokens": 4096, "top_k": 2, "tail": 0, "k": 4096, "n": 14336, "g": 8, "skew": 0.0, "out": "bf16"},
        # prompt processing at eight of 256 experts of very different popularity
        {"name": "product_many_experts", "op": "product", "tokens": 4096, "top_k": 8, "tail": 0, "k": 7168, "n": 2048, "g": 256, "skew": 1.1, "out": "bf16"},
        # training: a micro-batch of odd sizes where a quarter of the copies was not routed
        {"name": "permute_grad_small", "op": "permute_grad", "tokens": 61, "top_k": 3, "k": 1030, "drop": 0.25, "dtype": "f32"},
        # training: 4096 tokens of width 7168 at eight experts
        {"name": "permute_grad", "op": "permute_grad", "tokens": 4096, "top_k": 8, "k": 7168, "drop": 0.0, "dtype": "bf16"},
        {"name": "unpermute_grad_small", "op": "unpermute_grad", "tokens": 61, "top_k": 3, "k": 1030, "drop": 0.25, "dtype": "f32"},
        {"name": "unpermute_grad", "op": "unpermute_grad", "tokens": 4096, "top_k": 8, "k": 7168, "drop": 0.0, "dtype": "bf16"},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["quantize", "weights", "product", "product", "product", "permute_grad", "unpermute_grad"])
    if op == "quantize":
        return {"op": op, "rows": _log(rng, 1, 8192), "k": 32 * _log(rng, 1, 256), "dtype": rng.choice(["bf16", "f32"])}
    if op == "weights":
        g, n = _log(rng, 1, 16), _log(rng, 33, 14336)
        k = 32 * _log(rng, 1, 128)
        return {"op": op, "g": g, "k": k, "n": n, "dtype": rng.choice(["bf16", "bf16", "f32"])}
    if op == "product":
        g = rng.choice([1, 4, 8, 16, 60, 64, 128, 256])
        top_k = rng.randint(1, min(8, g))
        tokens = _log(rng, 1, 8192 // top_k)
        most = 3_000_000_000 // g          # elements of one expert's weights
        k = 32 * _log(rng, 4, 224)
        n = _log(rng, 64, max(65, min(14336, most // k)))
        n = n if rng.random() < 0.25 else -(-n // 16) * 16
        return {"op": op, "tokens": tokens, "top_k": top_k, "tail": rng.choice([0, 0, 0, rng.randint(1, 40)]), "k": k, "n": n, "g": g,
                "skew": rng.choice([0.0, 0.0, 0.8, 1.1]), "out": rng.choice(["bf16", "bf16", "f32"])}
    top_k = rng.randint(1, 8)
    return {"op": op, "tokens": _log(rng, 1, 32768 // top_k), "top_k": top_k, "k": rng.choice([_log(rng, 17, 7168), 8 * _log(rng, 8, 896)]),
            "drop": rng.choice([0.0, 0.0, 0.1]), "dtype": rng.choice(["bf16", "bf16", "f32"])}


# ---------------------------------------------------------------------------------------------
# inputs


def _panels(scale, rows):
    """[..., rows, k/32] scale bytes as [..., ceil(k/256), rows, 8], zero past k."""
    pad = -scale.shape[-1] % 8
    s = torch.nn.functional.pad(scale, (0, pad))
    s = s.reshape(*s.shape[:-1], -1, 8)
    return s.movedim(-3, -2).contiguous()


def _codes(x):
    """fp32 rows [rows, k] as 4-bit codes [rows, k/2] and scale bytes [rows, k/32]: inputs of the product cases."""
    rows, k = x.shape
    b = x.reshape(rows, k // 32, 32)
    e = (b.abs().amax(-1).view(torch.int32) >> 23) - 2
    e = e.clamp_min_(0)
    a = b * ((254 - e) << 23).view(torch.float32).unsqueeze(-1)
    s = a.signbit()
    a = a.abs_()
    c = torch.where(a < 2, torch.round(a * 2), torch.where(a < 4, torch.round(a) + 2, torch.round(a * 0.5) + 4)).clamp_max_(7).to(torch.uint8)
    c = (c | (s.to(torch.uint8) << 3)).reshape(rows, k // 2, 2)
    return c[..., 0] | (c[..., 1] << 4), e.to(torch.uint8)


def _activations(gen, rows, k):
    """Rows as a layer sees them: each channel has a size of its own, a few are much larger."""
    x = torch.randn(rows, k, device=DEV, generator=gen)
    c = torch.exp(0.5 * torch.randn(k, device=DEV, generator=gen))
    c = torch.where(torch.rand(k, device=DEV, generator=gen) < 0.01, 10 * c, c)
    return x * c


def _experts(gen, tokens, top_k, g, skew):
    """The top_k distinct experts of every token: normal scores, or popularity rank^-skew."""
    u = torch.rand(tokens, g, device=DEV, generator=gen).clamp_(1e-30, 1 - 1e-7)
    score = -torch.log(-torch.log(u))
    if skew:
        rank = torch.randperm(g, device=DEV, generator=gen).float() + 1
        score = score - skew * torch.log(rank)
    return score.topk(top_k, dim=1).indices


def prepare(case, seed):
    gen = torch.Generator(DEV)
    gen.manual_seed(int(seed))
    op, s = case["op"], {"op": case["op"]}
    if op == "quantize":
        s["x"] = _activations(gen, case["rows"], case["k"]).to(DT[case["dtype"]])
    elif op == "weights":
        g, k, n = case["g"], case["k"], case["n"]
        s["w"] = torch.empty(g, k, n, device=DEV, dtype=DT[case["dtype"]])
        for h in range(g):
            s["w"][h] = torch.randn(k, n, device=DEV, generator=gen) / math.sqrt(k)
    elif op == "product":
        k, n, g = case["k"], case["n"], case["g"]
        sizes = torch.bincount(_experts(gen, case["tokens"], case["top_k"], g, case["skew"]).reshape(-1), minlength=g)
        m = case["tokens"] * case["top_k"] + case["tail"]
        lhs, ls = _codes(_activations(gen, m, k))
        rhs = torch.empty(g, n, k // 2, device=DEV, dtype=torch.uint8)
        rs = torch.empty(g, n, k // 32, device=DEV, dtype=torch.uint8)
        for h in range(g):
            rhs[h], rs[h] = _codes(torch.randn(n, k, device=DEV, generator=gen) / math.sqrt(k))
        s |= {"lhs": lhs.view(FP4), "ls": _panels(ls, m), "rhs": rhs.view(FP4), "rs": _panels(rs, n), "sizes": sizes.to(torch.int32),
              "out": DT[case["out"]], "most": int(sizes.max())}
    else:
        tokens, top_k, k, dt = case["tokens"], case["top_k"], case["k"], DT[case["dtype"]]
        copies = tokens * top_k
        e = torch.randint(0, 256, (copies,), device=DEV, generator=gen)
        routed = torch.rand(copies, device=DEV, generator=gen) >= case["drop"]
        order = torch.argsort(torch.where(routed, e, 256), stable=True)
        total = int(routed.sum())
        s2c = torch.full((copies,), -1, device=DEV, dtype=torch.int32)
        s2c[:total] = order[:total].to(torch.int32)
        c2s = torch.full((copies,), -1, device=DEV, dtype=torch.int32)
        c2s[order[:total]] = torch.arange(total, device=DEV, dtype=torch.int32)
        s |= {"c2s": c2s, "s2c": s2c, "top_k": top_k}
        s["rows"] = torch.randn(copies, k, device=DEV, generator=gen).to(dt)
        if op == "unpermute_grad":
            s["dout"] = torch.randn(tokens, k, device=DEV, generator=gen).to(dt)
            s["weights"] = torch.softmax(torch.randn(tokens, top_k, device=DEV, generator=gen), 1)
    return s


# ---------------------------------------------------------------------------------------------
# the operators in plain operations


def _pow2(byte):
    """2^(byte - 127) in fp32 from its bits; 255 is NaN."""
    b = byte.to(torch.int32)
    bits = torch.where(b == 0, 0x00400000, torch.where(b == 255, 0x7FC00000, b << 23))
    return bits.to(torch.int32).view(torch.float32)


def _rounded(x):
    """fp32 blocks [..., 32] to the values that their 4-bit codes and scale stand for."""
    e = (x.abs().amax(-1, keepdim=True).view(torch.int32) >> 23)
    e = torch.where(e == 255, 255, (e - 2).clamp_min(0))
    a = x * ((254 - e) << 23).to(torch.int32).view(torch.float32)
    b = a.abs()
    step = torch.where(b < 2, 0.5, torch.where(b < 4, 1.0, 2.0))
    q = (torch.round(b / step) * step).clamp_max(6.0)
    return torch.copysign(q, a) * _pow2(e)


def _values(codes, scale):
    """Codes [..., rows, k/2] and scale panels [..., kp, rows, 8] to fp32 values [..., rows, k]."""
    table = torch.tensor([0, 0.5, 1, 1.5, 2, 3, 4, 6, -0.0, -0.5, -1, -1.5, -2, -3, -4, -6], device=DEV)
    c = codes.view(torch.uint8)
    c = torch.stack([c & 15, c >> 4], -1).to(torch.int32)
    v = table.index_select(0, c.reshape(-1)).reshape(*codes.shape[:-1], -1, 32)
    s = _pow2(scale.movedim(-3, -2).flatten(-2)[..., : v.shape[-2]])
    return (v * s.unsqueeze(-1)).flatten(-2)


def _product(s):
    lhs, rhs, sizes = _values(s["lhs"], s["ls"]), _values(s["rhs"], s["rs"]), s["sizes"].long()
    m, g, most = lhs.shape[0], rhs.shape[0], max(1, s["most"])
    end = torch.cumsum(sizes, 0)
    start = end - sizes
    slot = torch.arange(most, device=DEV)
    row = (start[:, None] + slot).clamp_max(m - 1)
    padded = lhs[row] * (slot < sizes[:, None])[..., None]
    full = torch.bmm(padded, rhs.transpose(1, 2).contiguous()).reshape(g * most, -1)
    r = torch.arange(m, device=DEV)
    h = torch.searchsorted(end, r, right=True)
    inside = (h < g)[:, None]
    h = h.clamp_max(g - 1)
    out = full[h * most + (r - start[h]).clamp(0, most - 1)]
    return torch.where(inside, out, 0.0).to(s["out"])


def run(s):
    op = s["op"]
    if own:
        import group_gemm_amd as G
        if op == "quantize":
            return G.mxfp4_dequantize(*G.mxfp4_quantize(s["x"]))
        if op == "weights":
            return G.mxfp4_dequantize(*G.mxfp4_quantize_weights(s["w"]))
        if op == "product":
            return G.ragged_dot_m_mxfp4(s["lhs"], s["rhs"], s["sizes"], s["ls"], s["rs"], out_dtype=s["out"])
        if op == "permute_grad":
            return G.moe_permute_grad(s["rows"], s["c2s"], s["top_k"])
        return G.moe_unpermute_grad(s["dout"], s["rows"], s["c2s"], s["s2c"], s["weights"])
    if op == "quantize":
        x = s["x"].float()
        return _rounded(x.reshape(x.shape[0], -1, 32)).reshape(x.shape).to(torch.bfloat16)
    if op == "weights":
        w = s["w"].float().transpose(1, 2).contiguous()
        return _rounded(w.reshape(w.shape[0], w.shape[1], -1, 32)).reshape(w.shape).to(torch.bfloat16)
    if op == "product":
        return _product(s)
    c2s, k = s["c2s"], s["rows"].shape[1]
    routed = (c2s >= 0)[:, None]
    rows = torch.where(routed, s["rows"][c2s.clamp_min(0)].float(), 0.0)
    if op == "permute_grad":
        return rows.reshape(-1, s["top_k"], k).sum(1).to(s["rows"].dtype)
    dout, s2c = s["dout"].float(), s["s2c"]
    dw = (rows.reshape(-1, s["top_k"], k) * dout[:, None]).sum(-1)
    at = s2c.clamp_min(0).long()
    dy = s["weights"].reshape(-1)[at][:, None] * dout[at // s["top_k"]]
    return torch.where((s2c >= 0)[:, None], dy, 0.0).to(s["rows"].dtype), dw


def _used(case):
    """Expected number of experts with a row."""
    g, p = case["g"], case["top_k"] / case["g"]
    return max(1.0, g if case["skew"] else g * (1 - (1 - p) ** case["tokens"]))


def work(case):
    op = case["op"]
    if op in ("quantize", "weights"):
        n = case["rows"] * case["k"] if op == "quantize" else case["g"] * case["k"] * case["n"]
        return {"bytes": n * ((4 if case["dtype"] == "f32" else 2) + 2), "flops": 2 * n}
    if op == "product":
        rows, k, n = case["tokens"] * case["top_k"], case["k"], case["n"]
        m = rows + case["tail"]
        b = (rows + _used(case) * n) * (k / 2 + k / 32) + m * n * (4 if case["out"] == "f32" else 2)
        return {"bytes": b, "flops": 2.0 * rows * k * n}
    e = 4 if case["dtype"] == "f32" else 2
    copies, k = case["tokens"] * case["top_k"], case["k"]
    kept = copies * (1 - case["drop"])
    if op == "permute_grad":
        return {"bytes": (kept + case["tokens"]) * k * e + 4 * copies, "flops": kept * k}
    return {"bytes": (kept + copies + case["tokens"]) * k * e + 16 * copies, "flops": 3 * kept * k}


# ---------------------------------------------------------------------------------------------
# the operators in 64 bits


def _exact_blocks(x):
    """Blocks [..., 32] in 64 bits: the nearest multiples of a power of two on the 4-bit grid, ties to the even code."""
    x = x.double()
    _, e = torch.frexp(x.abs().amax(-1, keepdim=True))
    e = (e - 3).clamp_min(-127)
    a = torch.ldexp(x.abs(), -e)
    q = torch.zeros_like(a)
    for at, even_above, gain in ((0.25, False, 0.5), (0.75, True, 0.5), (1.25, False, 0.5), (1.75, True, 0.5), (2.5, False, 1.0), (3.5, True, 1.0), (5.0, False, 2.0)):
        q += gain * ((a >= at) if even_above else (a > at))
    return torch.ldexp(q * torch.sign(x), e)


def _exact_values(codes, scale):
    """4-bit codes [rows, k/2] and scale bytes [rows, k/32] in 64 bits, by the format: sign, 2 exponent bits of bias 1, 1 bit."""
    rows, c = codes.shape[0], codes.view(torch.uint8).to(torch.int64)
    c = torch.stack([c % 16, c // 16], 2).reshape(rows, -1)
    e, f = (c % 8) // 2, (c % 2).double()
    v = torch.where(e == 0, f / 2, (1 + f / 2) * (2.0 ** (e - 1).double()))
    v = torch.where(c >= 8, -v, v)
    p = torch.tensor(2.0 ** (np.arange(256, dtype=np.float64) - 127), device=DEV)
    return (v.reshape(rows, -1, 32) * p[scale.long()][..., None]).reshape(rows, -1)


def exact(case, seed):
    s, op = prepare(case, seed), case["op"]
    if op == "quantize":
        return _exact_blocks(s["x"].reshape(case["rows"], -1, 32)).reshape(case["rows"], -1)
    if op == "weights":
        out = torch.empty(case["g"], case["n"], case["k"], device=DEV, dtype=torch.float64)
        for h in range(case["g"]):
            out[h] = _exact_blocks(s["w"][h].t().reshape(case["n"], -1, 32)).reshape(case["n"], -1)
        return out
    if op == "product":
        kb = case["k"] // 32
        ls = s["ls"].permute(1, 0, 2).reshape(s["lhs"].shape[0], -1)[:, :kb]
        x = _exact_values(s["lhs"], ls)
        out = torch.zeros(x.shape[0], case["n"], device=DEV, dtype=torch.float64)
        at = 0
        for h, size in enumerate(s["sizes"].tolist()):
            if size:
                w = _exact_values(s["rhs"][h], s["rs"][h].permute(1, 0, 2).reshape(case["n"], -1)[:, :kb])
                out[at:at + size] = x[at:at + size] @ w.t().contiguous()
            at += size
        return out
    c2s, rows = s["c2s"].tolist(), s["rows"].double()
    copies = torch.tensor([i for i, p in enumerate(c2s) if p >= 0], device=DEV)
    places = torch.tensor([p for p in c2s if p >= 0], device=DEV)
    tokens = copies // case["top_k"]
    if op == "permute_grad":
        return torch.zeros(case["tokens"], case["k"], device=DEV, dtype=torch.float64).index_add_(0, tokens, rows[places])
    dout, w = s["dout"].double(), s["weights"].double().reshape(-1)
    dy = torch.zeros_like(rows)
    dy[places] = w[copies, None] * dout[tokens]
    dw = torch.zeros_like(w)
    dw[copies] = (rows[places] * dout[tokens]).sum(1)
    return dy, dw.reshape(case["tokens"], case["top_k"])
