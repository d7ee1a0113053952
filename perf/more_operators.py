"""The 8-bit integer side of a decoder layer, case by case: what it computes in
plain torch operations, and the calls of this package that compute the same.

Four groups of operators, as a layer's rows pass through them:

* ``norm``: the residual stream plus a projection's rows, its RMS norm in 8 bits
  with a scale per row (read back as the values the codes stand for);
* ``gemm``: rows in 8 bits times a weight in 8 bits, with a scale per row and per
  output channel;
* ``mlp``: a dense MLP of those: norm, gate and up, silu(gate) * up in 8 bits,
  down;
* ``moe``: the router and the experts of a mixture layer for a few tokens.

A row of 8-bit codes stands for scale * code with scale = max|x| / 127, code =
x * (127 / max|x|) rounded half to even.
"""
import math
import random

import torch

own = False


# ------------------------------------------------------------------- cases
def listed():
    return [
        # one decode step's rows into the residual stream: pure latency (Qwen3-4B hidden size)
        dict(name="norm_1x2560", op="norm", m=1, n=2560, x32=True, r32=False),
        # prompts of several requests in a 27B-shaped layer, bf16 rows
        dict(name="norm_8190x5120", op="norm", m=8190, n=5120, x32=False, r32=False),
        # gate and up of one token, Qwen3-4B shapes: the weight's stream
        dict(name="gemm_1x19456x2560", op="gemm", m=1, n=19456, k=2560, y32=True),
        # down of a 17-row verify round, 27B shapes: few columns, long sums
        dict(name="gemm_17x5120x17408", op="gemm", m=17, n=5120, k=17408, y32=False),
        # an odd product: a small head over 33 rows
        dict(name="gemm_33x1001x777", op="gemm", m=33, n=1001, k=777, y32=True),
        # a short prompt through q, k and v of an 8B-shaped layer
        dict(name="gemm_301x6144x4096", op="gemm", m=301, n=6144, k=4096, y32=False),
        # a long prompt through a 27B-shaped projection
        dict(name="gemm_4096x17408x5120", op="gemm", m=4096, n=17408, k=5120, y32=False),
        # the dense MLP of a 6-row verify round (Qwen3-4B)
        dict(name="mlp_6x2560x9728", op="mlp", m=6, n=2560, f=9728),
        # the same of a prompt
        dict(name="mlp_1500x2560x9728", op="mlp", m=1500, n=2560, f=9728),
        # one token through 8 of 128 small experts
        dict(name="moe_1_8of128", op="moe", m=1, n=2048, f=768, e=128, top=8, norm=True),
        # a 6-row verify round through the same
        dict(name="moe_6_8of128", op="moe", m=6, n=2048, f=768, e=128, top=8, norm=True),
        # four requests of 8 rows through 2 of 8 large experts
        dict(name="moe_32_2of8", op="moe", m=32, n=4096, f=14336, e=8, top=2, norm=True),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def _size(rng, lo, hi):
    """A size over the logarithm of its range: half of them multiples of 128, the others any."""
    n = _log(rng, lo, hi)
    return max(128, n // 128 * 128) if rng.random() < 0.5 else n


def draw(rng):
    op = rng.choice(["gemm", "gemm", "gemm", "norm", "mlp", "moe", "moe"])
    if op == "norm":
        n = _size(rng, 64, 17408)
        return dict(op=op, m=_log(rng, 1, max(1, min(8190, 8190 * 5120 // n // 2))), n=n, x32=rng.random() < 0.5,
                    r32=rng.random() < 0.3)
    if op == "gemm":
        n, k = _size(rng, 64, 32768), _size(rng, 64, 17408)
        room = 4096 * 17408 * 5120 // (n * k)
        return dict(op=op, m=_log(rng, 1, max(1, min(8192, room))), n=n, k=k, y32=rng.random() < 0.5)
    if op == "mlp":
        n, f = _size(rng, 256, 5120), _size(rng, 256, 17408)
        room = 4096 * 17408 * 5120 // (3 * n * f)
        return dict(op=op, m=_log(rng, 1, max(1, min(4096, room))), n=n, f=f)
    e = rng.choice([4, 8, 16, 32, 60, 64, 128, 256])
    top, n = rng.randint(1, min(8, e)), _size(rng, 256, 4096)
    f = _size(rng, 128, max(129, min(8192, 8 * 4096 * 14336 // (e * n))))
    return dict(op=op, m=_log(rng, 1, max(1, min(64, 64 * 4096 * 14336 // (top * n * f)))), n=n, f=f, e=e, top=top,
                norm=rng.random() < 0.5)


# ------------------------------------------------------------------ inputs
def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed))
    return g


def _rows(m, n, dtype):
    """Rows of n values, their leading dimension padded to whole 16-byte pieces."""
    return torch.zeros(m, -(-n // 16) * 16, dtype=dtype, device="cuda")[:, :n]


def _normal(g, m, n, dtype, std=1.0, far=0.0):
    """Normal rows; `far` of the columns are ten times as large, as in a residual stream."""
    x = torch.empty((m, n), device="cuda").normal_(0.0, std, generator=g)
    if far:
        x *= torch.where(torch.empty(n, device="cuda").uniform_(generator=g) < far, 10.0, 1.0)
    out = _rows(m, n, dtype)
    out.copy_(x)
    return out


def _codes(g, *shape):
    """8-bit codes of normal values, and a scale for each row of them."""
    c = torch.empty(shape, device="cuda").normal_(0.0, 36.0, generator=g).round_().clamp_(-127, 127).to(torch.int8)
    return c, torch.empty(shape[:-1], device="cuda").uniform_(0.5, 1.5, generator=g) / (36.0 * math.sqrt(shape[-1]))


def _code_rows(g, m, n):
    c, out = _codes(g, m, n)[0], _rows(m, n, torch.int8)
    out.copy_(c)
    return out, torch.empty(m, device="cuda").uniform_(0.01, 0.05, generator=g)


def prepare(case, seed):
    g, op, m, n = _gen(seed), case["op"], case["m"], case["n"]
    s, bf = dict(case=case), torch.bfloat16
    if op in ("norm", "mlp"):
        s["x"] = _normal(g, m, n, torch.float32 if case.get("x32", True) else bf)
        s["res"] = _normal(g, m, n, torch.float32 if case.get("r32", False) else bf, 3.0, 1 / 256)
        s["w"] = 1 + 0.2 * torch.empty(n, device="cuda").normal_(generator=g)
        s["res_out"] = torch.empty_strided(s["res"].shape, s["res"].stride(), dtype=s["res"].dtype, device="cuda")
    if op == "norm":
        s["out"] = _rows(m, n, bf)
    elif op == "gemm":
        s["x8"], s["xs"] = _code_rows(g, m, case["k"])
        s["w8"], s["ws"] = _codes(g, n, case["k"])
        s["y"] = torch.empty(m, n, dtype=torch.float32 if case["y32"] else bf, device="cuda")
    elif op == "mlp":
        f = case["f"]
        s["gu8"], s["gus"] = _codes(g, 2 * f, n)
        s["dn8"], s["dns"] = _codes(g, n, f)
        s["y"] = torch.empty(m, n, dtype=bf, device="cuda")
    else:
        e, f = case["e"], case["f"]
        s["x"] = _normal(g, m, n, bf)
        top = s["x"].float().abs().amax(-1, keepdim=True)
        s["x8"], s["xs"] = _rows(m, n, torch.int8), (top / 127).view(-1)
        s["x8"].copy_((s["x"].float() * (127 / top)).round())
        s["router"] = _normal(g, e, n, bf, 1 / math.sqrt(n))
        (s["gate8"], s["gates"]), (s["up8"], s["ups"]) = _codes(g, e, f, n), _codes(g, e, f, n)
        s["dn8"], s["dns"] = _codes(g, e, n, f)
        s["ids"] = torch.empty(m, case["top"], dtype=torch.int32, device="cuda")
        s["wt"] = torch.empty(m, case["top"], device="cuda")
        s["y"] = torch.empty(m, n, dtype=bf, device="cuda")
    if own:
        s["calls"] = _calls(s)
    return s


def _calls(s):
    """The framework's calls of a pass, their arguments marshalled once, over weights packed once."""
    from speculative_decoding_verify_dspk_amd import binding
    c = s["case"]
    op, m, n = c["op"], c["m"], c["n"]
    codes = lambda k: (_rows(m, k, torch.int8), torch.empty(m, device="cuda"))  # noqa: E731
    if op in ("norm", "mlp"):
        c8, cs = codes(n)
        calls = [binding.prepare_add_rmsnorm(s["x"], s["res"], s["res_out"], s["w"], m, n, eps=1e-6, codes=c8, scales=cs)]
    if op == "norm":
        s["scales"] = cs
        return calls + [binding.prepare_i8_read(c8, cs, m, n, s["out"])]
    if op == "gemm":
        w = binding.Int8Weight(s["w8"], s["ws"])
        ws = binding.alloc_workspace(binding.i8_workspace_bytes(n, c["k"], m))
        return [binding.prepare_i8_gemm(w, s["x8"], s["xs"], m, s["y"], ws)]
    if op == "mlp":
        f = c["f"]
        gu, dn = binding.Int8Weight(s["gu8"], s["gus"]), binding.Int8Weight(s["dn8"], s["dns"])
        # of the products that are issued below
        wide = 2 * f if f % 8 == 0 else f
        need = max(binding.i8_workspace_bytes(wide, n, m), binding.i8_workspace_bytes(n, f, m))
        ws, (h8, hs) = binding.alloc_workspace(need), codes(f)
        # one product for both where up's columns start at a whole 16-byte piece
        if f % 8 == 0:
            both = _rows(m, 2 * f, torch.bfloat16)
            calls.append(binding.prepare_i8_gemm(gu, c8, cs, m, both, ws))
            gate, up = both[:, :f], both[:, f:]
        else:
            gw, uw = binding.Int8Weight(s["gu8"][:f], s["gus"][:f]), binding.Int8Weight(s["gu8"][f:], s["gus"][f:])
            gate, up = (_rows(m, f, torch.bfloat16) for _ in range(2))
            calls += [binding.prepare_i8_gemm(gw, c8, cs, m, gate, ws), binding.prepare_i8_gemm(uw, c8, cs, m, up, ws)]
        return calls + [binding.prepare_silu_mul(gate, up, m, f, codes=h8, scales=hs),
                        binding.prepare_i8_gemm(dn, h8, hs, m, s["y"], ws)]
    moe = binding.MoEWeights(binding.Int8Weight(s["gate8"], s["gates"]), binding.Int8Weight(s["up8"], s["ups"]),
                             binding.Int8Weight(s["dn8"], s["dns"]))
    ws = binding.alloc_workspace(binding.moe_workspace_bytes(n, c["f"], c["e"], m, c["top"]))
    return [binding.prepare_moe_route(s["x"], s["router"], m, s["ids"], s["wt"], ws, normalize=c["norm"]),
            binding.prepare_moe_mlp(moe, s["x8"], s["xs"], m, s["ids"], s["wt"], s["y"], ws)]


# ------------------------------------------------------------------ a pass
def run(s):
    op = s["case"]["op"]
    if own:
        for call in s["calls"]:
            call()
        if op == "norm":
            return s["res_out"], s["out"], s["scales"]
        if op == "gemm":
            return s["y"]
        if op == "mlp":
            return s["res_out"], s["y"]
        return s["ids"], s["wt"], s["y"]
    return {"norm": _norm, "gemm": _gemm, "mlp": _mlp, "moe": _moe}[op](s)


def _quantise(y):
    """Codes (held as floats) and scales of rows."""
    top = y.abs().amax(-1, keepdim=True)
    return torch.where(top > 0, (y * (127.0 / top)).round(), 0.0), top / 127.0


def _silu(g):
    return g / (1.0 + torch.exp(-g))


def _normed(s):
    t = s["x"].float() + s["res"].float()
    return t, t * torch.rsqrt(t.square().mean(-1, keepdim=True) + 1e-6) * s["w"]


def _norm(s):
    t, y = _normed(s)
    c, sc = _quantise(y)
    return t.to(s["res"].dtype), (c * sc).to(torch.bfloat16), sc.view(-1)


def _product(x, w):
    return torch.matmul(x, w.float().t())


def _gemm(s):
    return (_product(s["x8"].float(), s["w8"]) * s["xs"][:, None] * s["ws"]).to(s["y"].dtype)


def _mlp(s):
    t, y = _normed(s)
    c, sc = _quantise(y)
    gu = (_product(c, s["gu8"]) * sc * s["gus"]).to(torch.bfloat16).float()
    gate, up = gu.chunk(2, -1)
    h, hs = _quantise(_silu(gate) * up)
    return t.to(s["res"].dtype), (_product(h, s["dn8"]) * hs * s["dns"]).to(torch.bfloat16)


def _moe(s):
    c = s["case"]
    m, top = c["m"], c["top"]
    z = torch.matmul(s["x"].double(), s["router"].double().t())      # in 64 bits: which experts is a border
    z, ids = z.sort(dim=-1, descending=True, stable=True)
    p = torch.exp(z - z[:, :1])
    wt = (p[:, :top] / (p[:, :top] if c["norm"] else p).sum(-1, keepdim=True)).float()
    ids = ids[:, :top]
    e, x = ids.reshape(-1), s["x8"].float().repeat_interleave(top, 0).unsqueeze(-1)     # one row per token and slot
    xs = s["xs"].repeat_interleave(top)[:, None]
    gate = torch.matmul(s["gate8"][e].float(), x).squeeze(-1) * xs * s["gates"][e]
    up = torch.matmul(s["up8"][e].float(), x).squeeze(-1) * xs * s["ups"][e]
    h, hs = _quantise(_silu(gate) * up)
    y = torch.matmul(s["dn8"][e].float(), h.unsqueeze(-1)).squeeze(-1) * hs * s["dns"][e]
    y = (y.view(m, top, -1) * wt[..., None]).sum(1)
    return ids.int(), wt, y.to(torch.bfloat16)


# -------------------------------------------------------------------- work
def work(case):
    op, m, n = case["op"], case["m"], case["n"]
    if op == "norm":
        x, r = 4 if case["x32"] else 2, 4 if case["r32"] else 2
        # the codes are written, read back and written as bf16
        return dict(bytes=m * n * (x + 2 * r + 1 + 1 + 2) + 4 * n + 8 * m, flops=8 * m * n)
    if op == "gemm":
        k = case["k"]
        return dict(bytes=n * k + m * k + m * n * (4 if case["y32"] else 2) + 4 * (m + n), flops=2 * m * n * k)
    if op == "mlp":
        f = case["f"]
        return dict(bytes=3 * n * f + m * n * (4 + 2 + 2 + 2) + 4 * (4 * n + 2 * f), flops=6 * m * n * f)
    e, f, top = case["e"], case["f"], case["top"]
    used = e * (1 - (1 - top / e) ** m)                              # experts that some token chose, about
    return dict(bytes=int(used * (3 * n * f + 4 * (n + 2 * f)) + 2 * e * n + m * n * 5 + m * top * 8),
                flops=m * (6 * top * n * f + 2 * e * n))


# ------------------------------------------------------------------- exact
def _exact8(y):
    """Rows in 8 bits: the codes, and the step that they count."""
    step = y.abs().max(-1, keepdim=True).values / 127
    return torch.round(y / step.clamp(min=1e-300)), step


def exact(case, seed):
    s = prepare(case, seed)
    op, m, n = case["op"], case["m"], case["n"]
    if op in ("norm", "mlp"):
        t = s["x"].double() + s["res"].double()
        y = t / (t.pow(2).sum(-1, keepdim=True) / n + 1e-6).sqrt() * s["w"].double()
        c, step = _exact8(y)
        if op == "norm":
            return t, c * step, step.view(-1)
        wide = []
        for lo in range(0, 2 * case["f"], 4096):                     # a few columns of gate and up at a time
            w = s["gu8"][lo:lo + 4096].double() * s["gus"][lo:lo + 4096, None].double()
            wide.append(((c * step) @ w.T.contiguous()).to(torch.bfloat16).double())
        gate, up = torch.cat(wide, 1).split(case["f"], 1)
        c, step = _exact8(gate * torch.sigmoid(gate) * up)
        return t, (c @ s["dn8"].double().T.contiguous()) * step * s["dns"].double()
    if op == "gemm":
        x, outs = s["x8"].double() * s["xs"].double()[:, None], []
        for lo in range(0, n, 4096):
            outs.append(x @ (s["w8"][lo:lo + 4096].double() * s["ws"][lo:lo + 4096, None].double()).T.contiguous())
        return torch.cat(outs, 1)
    p = (s["x"].double() @ s["router"].double().T.contiguous()).softmax(-1).cpu()
    ids = [sorted(range(case["e"]), key=lambda j: (-r[j], j))[:case["top"]] for r in p.tolist()]
    wt = torch.stack([r[i] for r, i in zip(p, ids)])
    if case["norm"]:
        wt = wt / wt.sum(-1, keepdim=True)
    y = torch.zeros(m, n, dtype=torch.float64, device="cuda")
    x = s["x8"].double() * s["xs"].double()[:, None]
    for e in range(case["e"]):
        at = [(i, r.index(e)) for i, r in enumerate(ids) if e in r]
        if not at:
            continue
        rows = torch.tensor([i for i, _ in at], device="cuda")
        g = x[rows] @ (s["gate8"][e].double() * s["gates"][e, :, None].double()).T.contiguous()
        u = x[rows] @ (s["up8"][e].double() * s["ups"][e, :, None].double()).T.contiguous()
        c, step = _exact8(g * torch.sigmoid(g) * u)
        part = (c * step) @ (s["dn8"][e].double() * s["dns"][e, :, None].double()).T.contiguous()
        y.index_add_(0, rows, part * torch.stack([wt[i, j] for i, j in at]).cuda()[:, None])
    return torch.tensor(ids, dtype=torch.int32), wt, y
