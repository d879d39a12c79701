"""What is measured of the low-rank adapters and of the 8-bit activation checkpoints: the cases, their inputs, the
operators in plain torch operations and in 64 bits, and the calls that a user makes.

Operators (names and arguments as in group_gemm_amd):

* ``ragged_lora(x, a, b, group_sizes, base=..., row_group=..., scaling=..., v=...)``: low-rank adapters beside a
  shared projection, ``out[i] = base[i] + scaling[h] * (x[i] . a[h]^T) . b[h]^T`` with a [g, r, k] and b [g, n, r], where
  h is the adapter of row i: sorted rows with ``group_sizes``, or rows in any order with ``row_group`` (-1: none).
* ``ragged_lora_grad(x, v, dout, a, b, group_sizes, dbase=..., scaling=..., x_scale=...)``: its gradients dx, da and db,
  from x in 8 bits too.
* ``mxfp8_quantize(x)``, ``mxfp8_dequantize(codes, scale)``: rows [rows, k] to e4m3 codes with one power-of-two scale per
  32 elements along k, nothing clipped, and back.
* ``gated_act_mxfp8(gate, up, act)``: h = act(gate) * up with [gate | up] kept in 8 bits, and
  ``gated_act_mxfp8_grad(dh, codes, scale, act)``: dgate, dup and h from that checkpoint.
* ``ragged_dot_k(lhs, dout, group_sizes, lhs_scale=...)``: the experts' weight gradient from rows kept in 8 bits.
"""
import math

import torch

own = False
DEV = "cuda"
DT = {"bf16": torch.bfloat16, "f32": torch.float32}
E4M3 = torch.float8_e4m3fn


def listed():
    return [
        # one decoding token of one request, beside an up-projection: latency
        {"name": "lora_one_token", "op": "lora", "m": 1, "k": 4096, "n": 14336, "r": 16, "g": 8, "sorted": False, "none": 0.0, "save": False, "dtype": "bf16"},
        # a decoding batch of 96 requests in any order, each with one of 64 adapters, a tenth with none
        {"name": "lora_decode", "op": "lora", "m": 96, "k": 7168, "n": 2048, "r": 32, "g": 64, "sorted": False, "none": 0.1, "save": False, "dtype": "bf16"},
        # the training forward (and a prompt): 8192 rows sorted by one of eight adapters
        {"name": "lora_rows", "op": "lora", "m": 8192, "k": 4096, "n": 14336, "r": 64, "g": 8, "sorted": True, "none": 0.0, "save": True, "dtype": "bf16"},
        # training: gradients of 16 experts' adapters over 16384 tokens, the layer's input kept in 8 bits
        {"name": "lora_grad", "op": "lora_grad", "m": 16384, "k": 5120, "n": 8192, "r": 16, "g": 16, "none": 0.0, "x8": True, "dtype": "bf16", "grads": "f32"},
        # training: a small micro-batch of odd sizes, 32-bit, with rows past the last adapter's
        {"name": "lora_grad_odd", "op": "lora_grad", "m": 375, "k": 1030, "n": 515, "r": 11, "g": 5, "none": 0.1, "x8": False, "dtype": "f32", "grads": "f32"},
        # the input of an expert layer, kept in 8 bits and read back
        {"name": "rows", "op": "checkpoint", "kind": "rows", "m": 16384, "n": 5120, "act": "", "dtype": "bf16"},
        # the gated unit of an expert layer in training: 8192 rows of width 14336
        {"name": "gated", "op": "checkpoint", "kind": "gated", "m": 8192, "n": 14336, "act": "silu", "dtype": "bf16"},
        # the same for a handful of rows, 32-bit
        {"name": "gated_small", "op": "checkpoint", "kind": "gated", "m": 27, "n": 2880, "act": "gelu_tanh", "dtype": "f32"},
        # its backward pass from the checkpoint
        {"name": "gated_grad", "op": "gated_grad", "m": 8192, "n": 14336, "act": "silu", "dtype": "bf16"},
        {"name": "gated_grad_small", "op": "gated_grad", "m": 27, "n": 2880, "act": "gelu_tanh", "dtype": "f32"},
        # weight gradient of 16 experts of very different popularity from rows kept in 8 bits
        {"name": "wgrad", "op": "wgrad", "m": 16384, "k": 5120, "n": 8192, "g": 16, "tail": 0, "alpha": 0.5, "out": "f32"},
        # a small micro-batch at 32 experts, n without any alignment, rows past the last group
        {"name": "wgrad_odd", "op": "wgrad", "m": 387, "k": 2880, "n": 1447, "g": 32, "tail": 12, "alpha": 0.5, "out": "bf16"},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _rank(rng, g):
    r = rng.choice([4, 8, 16, 16, 32, 64, 128, rng.randint(1, 100)])
    return max(1, min(r, 2048 // g))


def draw(rng):
    op = rng.choice(["lora", "lora", "lora_grad", "lora_grad", "checkpoint", "gated_grad", "wgrad", "wgrad"])
    if op == "lora":
        g = rng.choice([1, 2, 8, 16, 64, 128])
        return {"op": op, "m": rng.choice([_log(rng, 1, 8192), rng.randint(1, 256)]), "k": rng.choice([_log(rng, 65, 7168), 64 * _log(rng, 1, 112)]),
                "n": rng.choice([_log(rng, 65, 14336), 64 * _log(rng, 1, 224)]), "r": min(_rank(rng, g), max(1, 512 // g)), "g": g,
                "sorted": rng.random() < 0.5, "none": rng.choice([0.0, 0.1, 0.5]), "save": rng.random() < 0.5, "dtype": rng.choice(["bf16", "bf16", "bf16", "f32"])}
    if op == "lora_grad":
        g, x8 = rng.choice([1, 2, 8, 16, 64]), rng.random() < 0.5
        return {"op": op, "m": _log(rng, 16, 16384), "k": 32 * _log(rng, 2, 160) if x8 else rng.choice([_log(rng, 65, 5120), 64 * _log(rng, 1, 80)]),
                "n": rng.choice([_log(rng, 65, 8192), 64 * _log(rng, 1, 128)]), "r": min(_rank(rng, g), max(1, 256 // g)), "g": g, "none": rng.choice([0.0, 0.1]),
                "x8": x8, "dtype": "bf16" if x8 else rng.choice(["bf16", "bf16", "f32"]), "grads": rng.choice(["f32", "f32", "bf16"])}
    if op == "checkpoint":
        kind = rng.choice(["rows", "gated"])
        return {"op": op, "kind": kind, "m": _log(rng, 1, 8192), "n": 32 * _log(rng, 1, 448 if kind == "gated" else 160), "act": rng.choice(["silu", "gelu_tanh"]),
                "dtype": rng.choice(["bf16", "f32"])}
    if op == "gated_grad":
        return {"op": op, "m": _log(rng, 1, 4096), "n": 32 * _log(rng, 1, 448), "act": rng.choice(["silu", "gelu_tanh"]), "dtype": rng.choice(["bf16", "f32"])}
    return {"op": op, "m": _log(rng, 16, 16384), "k": 32 * _log(rng, 2, 160), "n": rng.choice([_log(rng, 65, 4096), 64 * _log(rng, 1, 128)]),
            "g": rng.choice([1, 4, 16, 32]), "tail": rng.choice([0, 0, rng.randint(1, 15)]), "alpha": rng.choice([0.5, 1.5]), "out": rng.choice(["f32", "bf16"])}


# ---------------------------------------------------------------------------------------------
# inputs


def _activations(gen, rows, k):
    """Rows as a layer sees them: each channel has a size of its own, a few are much larger."""
    x = torch.randn(rows, k, device=DEV, generator=gen)
    c = torch.exp(0.5 * torch.randn(k, device=DEV, generator=gen))
    c = torch.where(torch.rand(k, device=DEV, generator=gen) < 0.01, 10 * c, c)
    return x * c


def _bytes8(b):
    """Scale bytes of fp32 blocks [..., 32]: the smallest power of two with which no value passes 448."""
    bits = b.abs().amax(-1).view(torch.int32)
    e = bits >> 23
    return torch.where(e == 255, 255, (e - 8 + ((bits & 0x7FFFFF) > 0x600000).to(torch.int32)).clamp_min(0))


def _power(e):
    """2^e in fp32 for e in [-127, 127], from its bits (2^-127 is a subnormal)."""
    return torch.where(e <= -127, 0x00400000, (e + 127) << 23).to(torch.int32).view(torch.float32)


def _codes8(x):
    """fp32 rows [rows, k] as e4m3 codes and scale bytes [rows, k/32]: inputs of the backward cases."""
    b = x.reshape(x.shape[0], -1, 32)
    e = _bytes8(b)
    return (b * _power(127 - e).unsqueeze(-1)).to(E4M3).reshape(x.shape), e.to(torch.uint8)


def _sizes(gen, m, g):
    """Rows of g groups of very different popularity, m in all."""
    p = torch.randn(g, device=DEV, generator=gen).square()
    c = torch.cumsum(p / p.sum(), 0)
    h = torch.searchsorted(c.clamp_max(1.0), torch.rand(m, device=DEV, generator=gen), right=True).clamp_max(g - 1)
    return torch.bincount(h, minlength=g).to(torch.int32)


def _adapters(gen, s, case):
    g, r, k, n, dt = case["g"], case["r"], case["k"], case["n"], DT[case["dtype"]]
    s["a"] = (torch.randn(g, r, k, device=DEV, generator=gen) / math.sqrt(k)).to(dt)
    s["b"] = (torch.randn(g, n, r, device=DEV, generator=gen) / math.sqrt(r)).to(dt)
    s["scaling"] = 2.0 ** torch.randint(-1, 2, (g,), device=DEV, generator=gen).float()


def prepare(case, seed):
    gen = torch.Generator(DEV)
    gen.manual_seed(int(seed))
    op, m, s = case["op"], case["m"], {"op": case["op"]}
    dt = DT[case.get("dtype", "bf16")]
    if op == "lora":
        _adapters(gen, s, case)
        s["x"] = _activations(gen, m, case["k"]).to(dt)
        s["base"] = torch.randn(m, case["n"], device=DEV, generator=gen).to(dt)
        s["sizes"] = s["rows"] = None
        if case["sorted"]:
            s["sizes"] = _sizes(gen, m - int(m * case["none"]), case["g"])
        else:
            h = torch.randint(0, case["g"], (m,), device=DEV, generator=gen)
            h = torch.where(torch.rand(m, device=DEV, generator=gen) < case["none"], -1, h)
            s["rows"] = h.to(torch.int32)
        s["save"] = case["save"]
    elif op == "lora_grad":
        _adapters(gen, s, case)
        x = _activations(gen, m, case["k"])
        s["xs"] = None
        s["x"] = x.to(dt)
        if case["x8"]:
            s["x"], s["xs"] = _codes8(x)
        s["v"] = torch.randn(m, case["r"], device=DEV, generator=gen)
        s["dout"] = torch.randn(m, case["n"], device=DEV, generator=gen).to(dt)
        s["dbase"] = torch.randn(m, case["k"], device=DEV, generator=gen).to(dt)
        s["sizes"] = _sizes(gen, m - int(m * case["none"]), case["g"])
        s["grads"] = DT[case["grads"]]
    elif op == "checkpoint":
        s["kind"], s["act"] = case["kind"], case["act"]
        s["x"] = _activations(gen, m, case["n"]).to(dt)
        if case["kind"] == "gated":
            s["up"] = _activations(gen, m, case["n"]).to(dt)
    elif op == "gated_grad":
        s["act"] = case["act"]
        x = torch.cat([_activations(gen, m, case["n"]), _activations(gen, m, case["n"])], 1)
        s["codes"], s["scale"] = _codes8(x)
        s["dh"] = torch.randn(m, case["n"], device=DEV, generator=gen).to(dt)
    else:
        s["lhs"], s["ls"] = _codes8(_activations(gen, m, case["k"]))
        s["dout"] = torch.randn(m, case["n"], device=DEV, generator=gen).to(torch.bfloat16)
        s["sizes"] = _sizes(gen, m - case["tail"], case["g"])
        s |= {"alpha": case["alpha"], "out": DT[case["out"]], "most": int(s["sizes"].max())}
    return s


# ---------------------------------------------------------------------------------------------
# the operators in plain operations


def _values8(codes, scale):
    """e4m3 codes [rows, k] and scale bytes [rows, k/32] to fp32 values."""
    p = _power(scale.to(torch.int32) - 127)
    return (codes.float().reshape(codes.shape[0], -1, 32) * p.unsqueeze(-1)).reshape(codes.shape)


def _members(s, m, g):
    """fp32 [m, g]: 1 where row i has adapter h."""
    if s.get("rows") is not None:
        h = s["rows"].long()
    else:
        h = torch.searchsorted(torch.cumsum(s["sizes"].long(), 0), torch.arange(m, device=DEV), right=True)
    return (h[:, None] == torch.arange(g, device=DEV)).float()


def _lora(s):
    a, b = s["a"].float(), s["b"].float()
    g, r, k = a.shape
    m, n = s["base"].shape
    member = _members(s, m, g)
    t = (s["x"].float() @ a.reshape(g * r, k).t()).reshape(m, g, r) * member[..., None]
    y = (t * s["scaling"][:, None]).reshape(m, g * r) @ b.permute(0, 2, 1).reshape(g * r, n)
    out = (s["base"].float() + y).to(s["base"].dtype)
    return (out, t.sum(1)) if s["save"] else out


def _lora_grad(s):
    a, b, dout = s["a"].float(), s["b"].float(), s["dout"].float()
    g, r, k = a.shape
    m, n = dout.shape
    x = _values8(s["x"], s["xs"]) if s["xs"] is not None else s["x"].float()
    member = _members(s, m, g) * s["scaling"]
    u = ((dout @ b.permute(1, 0, 2).reshape(n, g * r)).reshape(m, g, r) * member[..., None]).reshape(m, g * r)
    dx = (s["dbase"].float() + u @ a.reshape(g * r, k)).to(s["dbase"].dtype)
    da = (u.t() @ x).reshape(g, r, k)
    db = (dout.t() @ (s["v"][:, None, :] * member[..., None]).reshape(m, g * r)).reshape(n, g, r).permute(1, 0, 2)
    return dx, da.to(s["grads"]), db.to(s["grads"]).contiguous()


def _rounded8(x):
    """fp32 rows to the values that their 8-bit codes and scales stand for, in bfloat16 (which holds them)."""
    b = x.reshape(x.shape[0], -1, 32)
    e = _bytes8(b).unsqueeze(-1)
    return ((b * _power(127 - e)).to(E4M3).float() * _power(e - 127)).reshape(x.shape).to(torch.bfloat16)


def _gate(x, act):
    """act(x) and its derivative."""
    if act == "silu":
        p = 1 / (1 + torch.exp(-x))
        return x * p, p * (1 + x * (1 - p))
    c, d = math.sqrt(2 / math.pi), 0.044715
    t = torch.tanh(c * (x + d * x * x * x))
    return 0.5 * x * (1 + t), 0.5 * (1 + t) + 0.5 * x * (1 - t * t) * c * (1 + 3 * d * x * x)


def _wgrad(s):
    lhs, dout, sizes = _values8(s["lhs"], s["ls"]), s["dout"].float(), s["sizes"].long()
    m, most = lhs.shape[0], max(1, s["most"])
    start = torch.cumsum(sizes, 0) - sizes
    slot = torch.arange(most, device=DEV)
    row = (start[:, None] + slot).clamp_max(m - 1)
    left = (lhs[row] * (slot < sizes[:, None])[..., None]).transpose(1, 2).contiguous()
    return (s["alpha"] * torch.bmm(left, dout[row])).to(s["out"])


def run(s):
    op = s["op"]
    if own:
        import group_gemm_amd as G
        if op == "lora":
            v = torch.empty(s["x"].shape[0], s["a"].shape[1], device=DEV) if s["save"] else None
            out = G.ragged_lora(s["x"], s["a"], s["b"], s["sizes"], base=s["base"], row_group=s["rows"], scaling=s["scaling"], v=v)
            return (out, v) if s["save"] else out
        if op == "lora_grad":
            return G.ragged_lora_grad(s["x"], s["v"], s["dout"], s["a"], s["b"], s["sizes"], dbase=s["dbase"], scaling=s["scaling"], x_scale=s["xs"],
                                      grad_dtype=s["grads"])
        if op == "checkpoint":
            if s["kind"] == "rows":
                return G.mxfp8_dequantize(*G.mxfp8_quantize(s["x"]))
            h, codes, scale = G.gated_act_mxfp8(s["x"], s["up"], act=s["act"])
            return h, G.mxfp8_dequantize(codes, scale)
        if op == "gated_grad":
            return G.gated_act_mxfp8_grad(s["dh"], s["codes"], s["scale"], act=s["act"])
        return G.ragged_dot_k(s["lhs"], s["dout"], s["sizes"], lhs_scale=s["ls"], alpha=s["alpha"], out_dtype=s["out"])
    if op == "lora":
        return _lora(s)
    if op == "lora_grad":
        return _lora_grad(s)
    if op == "checkpoint":
        x = s["x"].float()
        if s["kind"] == "rows":
            return _rounded8(x)
        up = s["up"].float()
        return (_gate(x, s["act"])[0] * up).to(s["x"].dtype), _rounded8(torch.cat([x, up], 1))
    if op == "gated_grad":
        dh, dt = s["dh"].float(), s["dh"].dtype
        gate, up = _values8(s["codes"], s["scale"]).chunk(2, 1)
        f, d = _gate(gate, s["act"])
        return (dh * up * d).to(dt), (dh * f).to(dt), (f * up).to(dt)
    return _wgrad(s)


def _used(case):
    """Expected number of adapters with a row."""
    g = case["g"]
    return max(1.0, g * (1 - (1 - 1 / g) ** case["m"]))


def work(case):
    op, m, n = case["op"], case["m"], case["n"]
    e = 2 if case.get("dtype", "bf16") == "bf16" else 4
    if op == "lora":
        k, r = case["k"], case["r"]
        rows = m * (1 - case["none"])
        return {"bytes": rows * k * e + _used(case) * r * (k + n) * e + 2 * m * n * e + (4 * m * r if case["save"] else 0), "flops": 2.0 * rows * r * (k + n)}
    if op == "lora_grad":
        k, r, w = case["k"], case["r"], _used(case) * case["r"] * (case["k"] + case["n"])
        x = 33 / 32 if case["x8"] else e
        return {"bytes": m * k * x + m * n * e + 2 * m * k * e + 4 * m * r + w * (e + (4 if case["grads"] == "f32" else 2)), "flops": 4.0 * m * r * (k + n)}
    if op == "checkpoint":
        if case["kind"] == "rows":
            return {"bytes": m * n * (e + 2), "flops": 2.0 * m * n}
        return {"bytes": m * n * (3 * e + 4), "flops": 16.0 * m * n}
    if op == "gated_grad":
        return {"bytes": m * n * (4 * e + 33 / 16), "flops": 24.0 * m * n}
    k, rows = case["k"], m - case["tail"]
    return {"bytes": rows * (k * 33 / 32 + 2 * n) + case["g"] * k * n * (4 if case["out"] == "f32" else 2), "flops": 2.0 * rows * k * n}


# ---------------------------------------------------------------------------------------------
# the operators in 64 bits


def _two_to(e):
    """2^e in 64 bits from its bits, e in [-1022, 1023]."""
    return ((e.to(torch.int64) + 1023) << 52).view(torch.float64)


def _exact_values(codes, scale):
    """e4m3 codes and scale bytes in 64 bits, by the format: sign, 4 exponent bits of bias 7, 3 bits."""
    c = codes.view(torch.uint8).to(torch.int64)
    e, f = (c >> 3) % 16, (c % 8).double()
    v = torch.where(e == 0, f * 2.0 ** -9, (8 + f) * _two_to(e - 10))
    v = torch.where(c >= 128, -v, v).reshape(codes.shape[0], -1, 32)
    return (v * _two_to(scale.to(torch.int64) - 127)[..., None]).reshape(codes.shape)


def _exact_rounded(x):
    """The nearest values on the 8-bit grid, ties to even: steps of 2^-3 of a value's power of two, no finer than 2^-9 of the
    scale, which is the smallest power of two (2^-127 at least) with which the largest value is at most 448."""
    b = x.double().reshape(x.shape[0], -1, 32)
    most = b.abs().amax(-1, keepdim=True)
    _, e = torch.frexp(most)                       # most < 2^e, so 448 * 2^(e - 8) = 1.75 * 2^e holds it
    e = torch.where(448 * _two_to(e - 9) >= most, e - 9, e - 8).clamp_min(-127)
    _, p = torch.frexp(b)
    step = torch.maximum(p - 4, e - 9)
    return (torch.round(b * _two_to(-step)) * _two_to(step)).reshape(x.shape)


def _exact_gate(x, act):
    if act == "silu":
        p = torch.special.expit(x)
        return x * p, p + x * p * torch.special.expit(-x)
    z = math.sqrt(2 / math.pi) * (x + 0.044715 * x ** 3)
    t = torch.tanh(z)
    return x * (1 + t) / 2, (1 + t) / 2 + x / 2 / torch.cosh(z) ** 2 * math.sqrt(2 / math.pi) * (1 + 3 * 0.044715 * x ** 2)


def _rows_of(case, s):
    """The row numbers of every group."""
    if s.get("rows") is not None:
        h = s["rows"].tolist()
        return [[i for i in range(case["m"]) if h[i] == j] for j in range(case["g"])]
    sizes, at, found = s["sizes"].tolist(), 0, []
    for size in sizes:
        found.append(list(range(at, at + size)))
        at += size
    return found


def exact(case, seed):
    s, op, m = prepare(case, seed), case["op"], case["m"]
    if op == "lora":
        out, v = s["base"].double(), torch.zeros(m, case["r"], device=DEV, dtype=torch.float64)
        for h, rows in enumerate(_rows_of(case, s)):
            if rows:
                at = torch.tensor(rows, device=DEV)
                v[at] = s["x"][at].double() @ s["a"][h].double().t()
                out[at] += float(s["scaling"][h]) * (v[at] @ s["b"][h].double().t())
        return (out, v) if case["save"] else out
    if op == "lora_grad":
        x = _exact_values(s["x"], s["xs"]) if case["x8"] else s["x"].double()
        dx, da, db = s["dbase"].double(), torch.zeros_like(s["a"], dtype=torch.float64), torch.zeros_like(s["b"], dtype=torch.float64)
        for h, rows in enumerate(_rows_of(case, s)):
            if rows:
                at, w = slice(rows[0], rows[-1] + 1), float(s["scaling"][h])
                d = s["dout"][at].double()
                u = w * (d @ s["b"][h].double())
                dx[at] += u @ s["a"][h].double()
                da[h] = u.t() @ x[at]
                db[h] = w * (d.t() @ s["v"][at].double())
        return dx, da, db
    if op == "checkpoint":
        if case["kind"] == "rows":
            return _exact_rounded(s["x"])
        gate, up = s["x"].double(), s["up"].double()
        return _exact_gate(gate, case["act"])[0] * up, torch.cat([_exact_rounded(gate), _exact_rounded(up)], 1)
    if op == "gated_grad":
        x, n, dh = _exact_values(s["codes"], s["scale"]), case["n"], s["dh"].double()
        gate, up = x[:, :n], x[:, n:]
        f, d = _exact_gate(gate, case["act"])
        return dh * up * d, dh * f, f * up
    lhs, dout = _exact_values(s["lhs"], s["ls"]), s["dout"].double()
    out = torch.zeros(case["g"], case["k"], case["n"], device=DEV, dtype=torch.float64)
    for h, rows in enumerate(_rows_of(case, s)):
        if rows:
            out[h] = case["alpha"] * (lhs[rows[0]:rows[-1] + 1].t().contiguous() @ dout[rows[0]:rows[-1] + 1])
    return out
