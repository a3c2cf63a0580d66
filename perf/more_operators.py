"""Cases of the operators that train and adapt a block of packed layers:
attention over whole prompts, the residual stream's norms, low-rank adapters of
many requests beside a shared projection, and the gradient of the packed
product.

With `own` false, run() computes them from elementary torch operations in 32
bits; with `own` true it makes the library's calls.
"""
import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
DEV = "cuda"
EPS = 1e-6


# ---------------------------------------------------------------- the cases

def listed():
    return [
        # one short question before anything is generated: the call whose latency counts
        dict(name="attention, one short prompt", op="attention", lens="77", n_heads=32, n_kv=32, hd=128, dtype="bf16",
             lse=False),
        # a batch of prompts packed one behind the other, eight query heads to a kv head
        dict(name="attention, packed prompts", op="attention", lens="4096,2048,1371,2048", n_heads=64, n_kv=8, hd=128,
             dtype="bf16", lse=True),
        # a training step's batch of whole sequences
        dict(name="attention backward, four sequences", op="attention_backward", lens="2048x4", n_heads=32, n_kv=8,
             hd=128, dtype="bf16"),
        # examples of many lengths packed into one row, small heads
        dict(name="attention backward, ragged", op="attention_backward", lens="ragged:1:2900:13", n_heads=16, n_kv=4,
             hd=64, dtype="f16"),
        # the step between two sub-layers for one generated token
        dict(name="norm, one token", op="norm", m=1, d=8192, h="bf16", dtype="bf16", branch=True, post=False, gate=False,
             alpha=1.0),
        # a prompt through a block that norms, gates and scales what a sub-layer adds to a stream kept in 32 bits
        dict(name="norm, sandwich, 8192 tokens", op="norm", m=8192, d=5120, h="f32", dtype="bf16", branch=True, post=True,
             gate=True, alpha=0.22),
        # its gradients in a training step with an odd number of tokens
        dict(name="norm backward, 4095 tokens", op="norm_backward", m=4095, d=4096, h="bf16", dtype="bf16", branch=True,
             post=True, gate=True, alpha=0.22),
        # 48 requests generating, each through its own of 16 adapters or none
        dict(name="adapters, 48 requests", op="adapters", lens="1x48", n_adapters=16, d_in=8192, d_out=8192, rank=16,
             dtype="bf16", keep=False),
        # prompts of four requests; the backward pass follows
        dict(name="adapters, prompts, kept", op="adapters", lens="1500,1,1096,1499", n_adapters=3, d_in=5120, d_out=13824,
             rank=64, dtype="f16", keep=True),
        # a training step of two adapters, three sequences of one and one of the other
        dict(name="adapters backward, 8192 tokens", op="adapters_backward", lens="2048x4", n_adapters=2, d_in=4096,
             d_out=4096, rank=32, dtype="bf16"),
        # the gradient of an odd-sized batch through an output projection quantized in act order
        dict(name="linear backward, odd batch, act order", op="linear_backward", m=577, d_in=5120, d_out=5120, group=64,
             dtype="f16", perm=True, residual=True),
        # a training step through a frozen down projection
        dict(name="linear backward, 4096 tokens", op="linear_backward", m=4096, d_in=11008, d_out=4096, group=128,
             dtype="bf16", perm=False, residual=False),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _channels(rng, lo, hi):
    """Mostly multiples of 128, some only of 8."""
    return max(128, _log(rng, lo, hi) // 128 * 128) if rng.random() < 0.7 else max(8, _log(rng, lo, hi) // 8 * 8)


def draw(rng):
    op = rng.choice(["attention", "attention", "attention_backward", "norm", "norm_backward", "adapters", "adapters",
                     "adapters_backward", "linear_backward"])
    dtype = rng.choice(["bf16", "f16"])
    if op in ("attention", "attention_backward"):
        n_kv, rep, hd = rng.choice([1, 2, 4, 8]), rng.choice([1, 2, 3, 4, 8]), rng.choice([64, 128])
        n = rng.choice([1, 1, 2, 3, _log(rng, 2, 32)])
        lens = [_log(rng, 1, 4000) for _ in range(n)]
        # what it costs, and what the padded form of it holds
        while 2.0 * sum(v * v for v in lens) * n_kv * rep * hd * (5 if op.endswith("d") else 2) > 4e11 or \
                n * max(lens) ** 2 * n_kv * rep > 2.5e9:
            lens = [max(1, v * 3 // 4) for v in lens]
        c = dict(op=op, lens=",".join(map(str, lens)), n_heads=n_kv * rep, n_kv=n_kv, hd=hd, dtype=dtype)
        if op == "attention":
            c["lse"] = rng.random() < 0.5
        return c
    if op in ("norm", "norm_backward"):
        d = rng.choice([_log(rng, 64, 16384) // 8 * 8, _log(rng, 64, 16384), 128 * _log(rng, 1, 128)])
        m = _log(rng, 1 if op == "norm" else 8, max(8, min(16384, 40000000 // d)))
        branch = rng.random() < 0.85
        return dict(op=op, m=m, d=d, h=rng.choice([dtype, dtype, "f32"]), dtype=dtype, branch=branch,
                    post=branch and rng.random() < 0.4, gate=branch and rng.random() < 0.3,
                    alpha=rng.choice([1.0, 1.0, 0.22]) if branch else 1.0)
    if op in ("adapters", "adapters_backward"):
        n = _log(rng, 1, 64)
        one = op == "adapters" and rng.random() < 0.5
        lens = [1] * n if one else [_log(rng, 1, max(1, 8192 // n)) for _ in range(n)]
        c = dict(op=op, lens=",".join(map(str, lens)), n_adapters=_log(rng, 1, 32 if one else 6),
                 d_in=_channels(rng, 128, 8192), d_out=_channels(rng, 64, 11008), rank=rng.choice([8, 16, 16, 32, 64, 128]),
                 dtype=dtype)
        if op == "adapters":
            c["keep"] = rng.random() < 0.4
        # the padded form holds every sequence at the longest one's length
        while n * max(lens) * (c["d_in"] + c["d_out"]) > 1.5e9 or sum(lens) * (c["d_in"] + c["d_out"]) > 1e8:
            lens = [max(1, v * 3 // 4) for v in lens]
            c["lens"] = ",".join(map(str, lens))
        return c
    c = dict(op=op, m=_log(rng, 1, 8192), d_in=_channels(rng, 128, 13824), d_out=_channels(rng, 128, 11008),
             group=rng.choice([32, 64, 128, 128, -1]), dtype=dtype, perm=rng.random() < 0.3, residual=rng.random() < 0.5)
    while 2.0 * c["m"] * c["d_in"] * c["d_out"] > 3.7e11:
        c["m"] = c["m"] // 2
    return c


def _lens(text):
    """"3,4" -> [3, 4]; "1x48" -> 48 ones; "ragged:1:2900:13" -> 13 lengths from 1 to 2900, spread over their logarithm."""
    if text.startswith("ragged:"):
        lo, hi, n = map(int, text.split(":")[1:])
        return [int(round(lo * (hi / lo) ** (((5 * i) % n) / (n - 1)))) for i in range(n)]
    if "x" in text:
        v, n = map(int, text.split("x"))
        return [v] * n
    return [int(v) for v in text.split(",")]


# ---------------------------------------------------------------- what is in hand before the call

def _gen(seed):
    return torch.Generator(device=DEV).manual_seed(seed)


def _normal(g, shape, dtype, std=1.0):
    return (torch.randn(shape, generator=g, device=DEV) * std).to(dtype)


def _hidden(g, m, d, dtype, std=1.0):
    """Normal channels, one in 200 ten times as large, as a hidden state has them."""
    x = torch.randn((m, d), generator=g, device=DEV) * std
    x[:, torch.randperm(d, generator=g, device=DEV)[: max(1, d // 200)]] *= 10
    return x.to(dtype)


def _packed_weight(g, d_out, d_in, group):
    """A weight of N(0, 0.02) on its min-max 4-bit grid: packed codes [d_out, d_in/8], scales and zero points."""
    G = d_in if group == -1 else group
    ng = -(-d_in // G)
    w = torch.randn((d_out, ng * G), generator=g, device=DEV) * 0.02
    w[:, d_in:] = 0
    w = w.view(d_out, ng, G)
    lo, hi = w.amin(2), w.amax(2)
    scales = (hi - lo) / 15
    zeros = torch.round(-lo / scales)
    codes = (torch.round(w / scales[:, :, None]) + zeros[:, :, None]).clamp_(0, 15).to(torch.int32)
    codes = codes.view(d_out, ng * G)[:, :d_in].reshape(d_out, d_in // 8, 8)
    packed = codes[:, :, 0].clone()
    for k in range(1, 8):
        packed |= codes[:, :, k] << (4 * k)
    return dict(packed=packed, scales=scales.contiguous(), zeros=zeros.to(torch.int32).contiguous(), group=group)


def _sequences(s, text):
    lens = _lens(text)
    starts = [0]
    for n in lens:
        starts.append(starts[-1] + n)
    s.update(lens=lens, tokens=starts[-1], q_start=torch.tensor(starts, dtype=torch.int32, device=DEV))


def prepare(case, seed):
    g = _gen(seed)
    op, dt = case["op"], DTYPES[case["dtype"]]
    s = dict(case=case)
    if op in ("attention", "attention_backward"):
        _sequences(s, case["lens"])
        T, H, n_kv, hd = s["tokens"], case["n_heads"], case["n_kv"], case["hd"]
        # a fused projection's rows hold queries, keys and values side by side; a few key channels are large
        row = torch.randn((T, H + 2 * n_kv, hd), generator=g, device=DEV)
        row[:, H:H + n_kv, : hd // 32] *= 4
        row = row.to(dt)
        s["q"], s["k"], s["v"] = row[:, :H], row[:, H:H + n_kv], row[:, H + n_kv:]
        if op == "attention_backward":
            s["do"] = _normal(g, (T, H, hd), dt, 0.01)
            out, s["lse"] = _attend(s)
            s["out"] = out.to(dt)
    elif op in ("norm", "norm_backward"):
        m, d, ht = case["m"], case["d"], DTYPES[case["h"]]
        s["r"] = _hidden(g, m, d, ht)
        s["b"] = _hidden(g, m, d, dt, 0.3) if case["branch"] else None
        s["gamma"] = 1 + 0.2 * torch.randn(d, generator=g, device=DEV)
        s["post"] = 0.3 + 0.1 * torch.randn(d, generator=g, device=DEV) if case["post"] else None
        s["gate"] = torch.randn(d, generator=g, device=DEV) if case["gate"] else None
        if op == "norm_backward":
            # r stands for the stream that the forward pass wrote
            s["dy"], s["dh"] = _normal(g, (m, d), dt, 0.01), _normal(g, (m, d), ht, 0.01)
    elif op in ("adapters", "adapters_backward"):
        _sequences(s, case["lens"])
        T, n, r = s["tokens"], case["n_adapters"], case["rank"]
        s["a"] = _normal(g, (n, r, case["d_in"]), dt, case["d_in"] ** -0.5)
        s["b"] = _normal(g, (n, case["d_out"], r), dt, 0.02)
        s["scale"] = 0.5 + 2 * torch.rand(n, generator=g, device=DEV)
        # one sequence in eight goes without an adapter
        which = torch.randint(0, n, (len(s["lens"]),), generator=g, device=DEV)
        none = torch.rand(len(s["lens"]), generator=g, device=DEV) < (0.125 if len(s["lens"]) > 4 else 0.0)
        s["adapter"] = torch.where(none, -1, which).to(torch.int32)
        s["x"] = _hidden(g, T, case["d_in"], dt)
        if op == "adapters":
            s["r"] = _normal(g, (T, case["d_out"]), dt)
        else:
            s["dy"], s["r"] = _normal(g, (T, case["d_out"]), dt, 0.01), _normal(g, (T, case["d_in"]), dt, 0.01)
            s["s"] = _low(s, s["x"], s["a"])
    else:
        s["w"] = _packed_weight(g, case["d_out"], case["d_in"], case["group"])
        s["perm"] = torch.randperm(case["d_in"], generator=g, device=DEV).to(torch.int32) if case["perm"] else None
        s["dy"] = _normal(g, (case["m"], case["d_out"]), dt, 0.01)
        s["r"] = _normal(g, (case["m"], case["d_in"]), dt, 0.01) if case["residual"] else None
    if own:
        _handles(s)
    return s


def _handles(s):
    """The library's descriptors and the output and scratch buffers a program keeps."""
    import post_weight_quantization_29_amd as P
    case = s["case"]
    op, dt = case["op"], DTYPES[case["dtype"]]
    new = lambda *shape, dtype=dt: torch.empty(shape, dtype=dtype, device=DEV)  # noqa: E731
    scratch = lambda n: new(max(1, n), dtype=torch.uint8)  # noqa: E731
    f32 = torch.float32
    if op == "attention":
        s["o"] = new(s["tokens"], case["n_heads"], case["hd"])
        s["l"] = new(s["tokens"], case["n_heads"], dtype=f32) if case["lse"] else None
    elif op == "attention_backward":
        s["dq"] = new(s["tokens"], case["n_heads"], case["hd"])
        s["dk"], s["dv"] = new(s["tokens"], case["n_kv"], case["hd"]), new(s["tokens"], case["n_kv"], case["hd"])
        s["ws"] = scratch(P.gptq_prompt_attention_backward_workspace_size(s["tokens"], case["n_heads"]))
    elif op == "norm":
        s["h"] = new(case["m"], case["d"], dtype=DTYPES[case["h"]]) if case["branch"] else None
        s["y"] = new(case["m"], case["d"])
    elif op == "norm_backward":
        s["dr"] = new(case["m"], case["d"], dtype=DTYPES[case["h"]])
        s["db"] = new(case["m"], case["d"]) if case["branch"] else None
        s["dgamma"] = new(case["d"], dtype=f32)
        s["dpost"] = new(case["d"], dtype=f32) if case["post"] else None
        s["dgate"] = new(case["d"], dtype=f32) if case["gate"] else None
        s["ws"] = scratch(P.gptq_residual_rmsnorm_backward_workspace_size(case["m"], case["d"]))
    elif op in ("adapters", "adapters_backward"):
        s["set"] = P.LoRASet(s["a"], s["b"], s["scale"])
        if op == "adapters":
            s["y"] = new(s["tokens"], case["d_out"])
            s["low"] = new(s["tokens"], case["rank"], dtype=f32) if case["keep"] else None
            s["ws"] = scratch(P.gptq_lora_workspace_size(s["tokens"], s["set"]))
        else:
            s["dx"] = new(s["tokens"], case["d_in"])
            s["da"] = new(case["n_adapters"], case["rank"], case["d_in"], dtype=f32)
            s["db"] = new(case["n_adapters"], case["d_out"], case["rank"], dtype=f32)
            s["ws"] = scratch(P.gptq_lora_backward_workspace_size(s["tokens"], s["set"]))
    else:
        s["h"] = P.W4Weight(s["w"]["packed"], s["w"]["scales"], s["w"]["zeros"], s["w"]["group"], s["perm"])
        s["dx"] = new(case["m"], case["d_in"])
        s["ws"] = scratch(P.gptq_w4_linear_backward_workspace_size(case["m"], s["h"]))


# ---------------------------------------------------------------- one pass

def run(s):
    if own:
        return _run_own(s)
    return {"attention": _attention, "attention_backward": _attention_backward, "norm": _norm,
            "norm_backward": _norm_backward, "adapters": _adapters, "adapters_backward": _adapters_backward,
            "linear_backward": _linear_backward}[s["case"]["op"]](s)


def _run_own(s):
    import post_weight_quantization_29_amd as P
    case = s["case"]
    op = case["op"]
    if op == "attention":
        P.gptq_prompt_attention(s["q"], s["k"], s["v"], s["q_start"], max(s["lens"]), s["o"], lse=s["l"])
        return {"out": s["o"], "lse": s["l"]} if case["lse"] else {"out": s["o"]}
    if op == "attention_backward":
        P.gptq_prompt_attention_backward(s["do"], s["q"], s["k"], s["v"], s["out"], s["lse"], s["q_start"], max(s["lens"]),
                                         s["dq"], s["dk"], s["dv"], ws=s["ws"])
        return {"dq": s["dq"], "dk": s["dk"], "dv": s["dv"]}
    if op == "norm":
        P.gptq_residual_rmsnorm(s["r"], s["y"], B=s["b"], H=s["h"], gamma=s["gamma"], post_gamma=s["post"], gate=s["gate"],
                                alpha=case["alpha"], eps=EPS)
        return {"h": s["h"], "y": s["y"]} if case["branch"] else {"y": s["y"]}
    if op == "norm_backward":
        P.gptq_residual_rmsnorm_backward(s["dy"], s["r"], s["dr"], dH=s["dh"], B=s["b"], dB=s["db"], gamma=s["gamma"],
                                         post_gamma=s["post"], gate=s["gate"], alpha=case["alpha"], eps=EPS,
                                         dgamma=s["dgamma"], dpost_gamma=s["dpost"], dgate=s["dgate"], ws=s["ws"])
        return {k: s[k] for k in ("dr", "db", "dgamma", "dpost", "dgate") if s[k] is not None}
    if op == "adapters":
        P.gptq_lora(s["x"], s["set"], s["q_start"], s["adapter"], s["y"], R=s["r"], S=s["low"], ws=s["ws"])
        return {"y": s["y"], "s": s["low"]} if case["keep"] else {"y": s["y"]}
    if op == "adapters_backward":
        P.gptq_lora_backward(s["dy"], s["x"], s["s"], s["set"], s["q_start"], s["adapter"], dX=s["dx"], R=s["r"], dA=s["da"],
                             dB=s["db"], ws=s["ws"])
        return {"dx": s["dx"], "da": s["da"], "db": s["db"]}
    P.gptq_w4_linear_backward(s["dy"], s["h"], s["dx"], R=s["r"], ws=s["ws"])
    return s["dx"]


def _rows(s):
    """[sequences, longest]: each token's row, and whether it is one."""
    start = s["q_start"].long()
    i = torch.arange(max(s["lens"]), device=DEV)
    return (start[:-1, None] + i).clamp(max=s["tokens"] - 1), i < (start[1:] - start[:-1])[:, None]


def _padded(x, rows, is_one):
    return torch.where(is_one.view(is_one.shape + (1,) * (x.dim() - 1)), x.float()[rows], 0.0)


def _scores(s, rows, is_one):
    """The queries, keys and values of each sequence, [sequences, kv heads, rows, hd], and the probabilities' logarithms' parts."""
    case = s["case"]
    n, most = rows.shape
    n_kv, hd = case["n_kv"], case["hd"]
    q = _padded(s["q"], rows, is_one).view(n, most, n_kv, -1, hd).permute(0, 2, 3, 1, 4).flatten(2, 3)
    k, v = (_padded(s[x], rows, is_one).transpose(1, 2) for x in "kv")
    score = q @ k.transpose(2, 3) / math.sqrt(hd)
    i = torch.arange(most, device=DEV)
    seen = (i[None] <= i[:, None]).repeat(case["n_heads"] // n_kv, 1)
    score = score.masked_fill_(~seen, float("-inf"))
    top = score.amax(-1, keepdim=True)
    p = score.sub_(top).exp_()
    total = p.sum(-1, keepdim=True)
    return q, k, v, p.div_(total), top + torch.log(total)


def _heads_back(x, case, is_one):
    """[sequences, kv heads, heads of each * longest, ...] -> [tokens, heads, ...]"""
    n, n_kv, rows = x.shape[:3]
    most = is_one.shape[1]
    x = x.reshape((n, n_kv, rows // most, most) + x.shape[3:])
    x = x.permute((0, 3, 1, 2) + tuple(range(4, x.dim()))).flatten(2, 3)
    return x[is_one]


def _attend(s):
    rows, is_one = _rows(s)
    q, k, v, p, lse = _scores(s, rows, is_one)
    return _heads_back(p @ v, s["case"], is_one), _heads_back(lse, s["case"], is_one)[..., 0].contiguous()


def _attention(s):
    out, lse = _attend(s)
    out = out.to(DTYPES[s["case"]["dtype"]])
    return {"out": out, "lse": lse} if s["case"]["lse"] else {"out": out}


def _attention_backward(s):
    case, dt = s["case"], DTYPES[s["case"]["dtype"]]
    rows, is_one = _rows(s)
    q, k, v, p, _ = _scores(s, rows, is_one)
    n, most = rows.shape
    do = _padded(s["do"], rows, is_one).view(n, most, case["n_kv"], -1, case["hd"]).permute(0, 2, 3, 1, 4).flatten(2, 3)
    dv = p.transpose(2, 3) @ do
    dp = do @ v.transpose(2, 3)
    ds = p * (dp - (p * dp).sum(-1, keepdim=True)) / math.sqrt(case["hd"])
    dq, dk = ds @ k, ds.transpose(2, 3) @ q
    return {"dq": _heads_back(dq, case, is_one).to(dt), "dk": dk.transpose(1, 2)[is_one].to(dt),
            "dv": dv.transpose(1, 2)[is_one].to(dt)}


def _unit(x):
    """x / sqrt(mean x^2 + eps), and that factor."""
    r = 1 / torch.sqrt((x * x).mean(-1, keepdim=True) + EPS)
    return x * r, r


def _branch(s):
    """What the sub-layer adds before gate and scale; its norm's parts where it has one."""
    b = s["b"].float()
    if s["post"] is None:
        return b, None, None
    unit, r = _unit(b)
    return unit * s["post"], unit, r


def _norm(s):
    case = s["case"]
    h = s["r"].float()
    if case["branch"]:
        b = _branch(s)[0]
        h = h + case["alpha"] * (b if s["gate"] is None else s["gate"] * b)
    y = (_unit(h)[0] * s["gamma"]).to(DTYPES[case["dtype"]])
    return {"h": h.to(DTYPES[case["h"]]), "y": y} if case["branch"] else {"y": y}


def _norm_backward(s):
    case = s["case"]
    dy = s["dy"].float()
    unit, r = _unit(s["r"].float())
    g = dy * s["gamma"]
    dh = s["dh"].float() + r * (g - unit * (g * unit).mean(-1, keepdim=True))
    out = {"dr": dh.to(DTYPES[case["h"]]), "dgamma": (dy * unit).sum(0)}
    if case["branch"]:
        b, unit_b, r_b = _branch(s)
        db = case["alpha"] * (dh if s["gate"] is None else s["gate"] * dh)
        if s["gate"] is not None:
            out["dgate"] = case["alpha"] * (dh * b).sum(0)
        if s["post"] is not None:
            out["dpost"] = (db * unit_b).sum(0)
            g = db * s["post"]
            db = r_b * (g - unit_b * (g * unit_b).mean(-1, keepdim=True))
        out["db"] = db.to(DTYPES[case["dtype"]])
    return out


def _chosen(s):
    """Each sequence's adapter and its scale, 0 where it has none."""
    has = s["adapter"] >= 0
    at = s["adapter"].clamp(min=0).long()
    return at, torch.where(has, s["scale"][at], 0.0), has


def _low(s, x, a):
    """x A^T of each token's adapter, [tokens, rank] (0 without one)."""
    rows, is_one = _rows(s)
    at, _, has = _chosen(s)
    low = _padded(x, rows, is_one) @ a.float()[at].transpose(1, 2)
    return (low * has[:, None, None])[is_one].contiguous()


def _adapters(s):
    rows, is_one = _rows(s)
    at, scale, _ = _chosen(s)
    low = _low(s, s["x"], s["a"])
    d = _padded(low, rows, is_one) @ s["b"].float()[at].transpose(1, 2)
    y = (s["r"].float() + (d * scale[:, None, None])[is_one]).to(s["r"].dtype)
    return {"y": y, "s": low} if s["case"]["keep"] else {"y": y}


def _adapters_backward(s):
    rows, is_one = _rows(s)
    at, scale, _ = _chosen(s)
    dy = _padded(s["dy"], rows, is_one) * scale[:, None, None]
    ds = dy @ s["b"].float()[at]
    dx = (s["r"].float() + (ds @ s["a"].float()[at])[is_one]).to(s["r"].dtype)
    da = torch.zeros(s["a"].shape, device=DEV).index_add_(0, at, ds.transpose(1, 2) @ _padded(s["x"], rows, is_one))
    db = torch.zeros(s["b"].shape, device=DEV).index_add_(0, at, dy.transpose(1, 2) @ _padded(s["s"], rows, is_one))
    return {"dx": dx, "da": da, "db": db}


def _dense(w, dtype):
    """The weight that the packed layer stands for: scale * (code - zero), rounded to the activations' type; as fp32."""
    shifts = torch.arange(0, 32, 4, device=DEV, dtype=torch.int32)
    codes = ((w["packed"][..., None] >> shifts) & 15).flatten(-2)
    d_in = codes.shape[1]
    G = d_in if w["group"] == -1 else w["group"]
    of = torch.arange(d_in, device=DEV) // G
    return (w["scales"][:, of] * (codes - w["zeros"][:, of]).float()).to(dtype).float()


def _linear_backward(s):
    dx = s["dy"].float() @ _dense(s["w"], s["dy"].dtype)
    if s["perm"] is not None:
        dx = torch.empty_like(dx).index_copy_(1, s["perm"].long(), dx)
    if s["r"] is not None:
        dx = dx + s["r"].float()
    return dx.to(s["dy"].dtype)


# ---------------------------------------------------------------- what a pass cannot do without

def work(case):
    op = case["op"]
    if op in ("attention", "attention_backward"):
        lens = _lens(case["lens"])
        seen, T = sum(n * (n + 1) // 2 for n in lens), sum(lens)
        q, kv = 2 * T * case["n_heads"] * case["hd"], 2 * T * case["n_kv"] * case["hd"]
        if op == "attention":
            return {"bytes": 2 * q + 2 * kv + (4 * T * case["n_heads"] if case["lse"] else 0),
                    "flops": 4 * seen * case["n_heads"] * case["hd"]}
        return {"bytes": 4 * q + 4 * kv + 4 * T * case["n_heads"], "flops": 10 * seen * case["n_heads"] * case["hd"]}
    if op in ("norm", "norm_backward"):
        n, hb = case["m"] * case["d"], 4 if case["h"] == "f32" else 2
        if op == "norm":
            return {"bytes": n * (hb + 2 + (hb + 2 if case["branch"] else 0)), "flops": 10 * n}
        return {"bytes": n * (3 * hb + 2 + (4 if case["branch"] else 0)), "flops": 25 * n}
    if op in ("adapters", "adapters_backward"):
        lens, both = _lens(case["lens"]), case["d_in"] + case["d_out"]
        T, sets = sum(lens), 2 * min(case["n_adapters"], len(lens)) * case["rank"] * both
        if op == "adapters":
            return {"bytes": sets + 2 * T * (case["d_in"] + 2 * case["d_out"]) + (4 * T * case["rank"] if case["keep"] else 0),
                    "flops": 2 * T * case["rank"] * both}
        return {"bytes": sets + 4 * case["n_adapters"] * case["rank"] * both + 2 * T * (3 * case["d_in"] + case["d_out"])
                + 4 * T * case["rank"], "flops": 4 * T * case["rank"] * both}
    G = case["d_in"] if case["group"] == -1 else case["group"]
    weight = case["d_out"] * (case["d_in"] // 2 + 8 * -(-case["d_in"] // G))
    return {"bytes": weight + 2 * case["m"] * (case["d_out"] + case["d_in"] * (2 if case["residual"] else 1))
            + (4 * case["d_in"] if case["perm"] else 0), "flops": 2 * case["m"] * case["d_in"] * case["d_out"]}


# ---------------------------------------------------------------- the definitions in 64 bits

def _attention64(q, k, v, rep):
    """One sequence: q [heads, n, hd], k and v [kv heads, n, hd]; the outputs and the scores' log-sum."""
    n = q.shape[1]
    score = torch.matmul(q, k.repeat_interleave(rep, 0).transpose(1, 2)) * q.shape[2] ** -0.5
    later = torch.ones((n, n), dtype=torch.bool, device=DEV).triu(1)
    score = score.masked_fill(later, -math.inf)
    return torch.matmul(torch.softmax(score, -1), v.repeat_interleave(rep, 0)), torch.logsumexp(score, -1)


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op in ("attention", "attention_backward"):
        rep, back = case["n_heads"] // case["n_kv"], op == "attention_backward"
        names = ("dq", "dk", "dv") if back else ("out", "lse")
        found = {x: [] for x in names}
        for t0, n in zip(s["q_start"].tolist(), s["lens"]):
            parts = {x: [] for x in names}
            for h in range(case["n_kv"]):          # a kv head and its query heads at a time
                at = [s[x][t0:t0 + n].double().transpose(0, 1) for x in "qkv"]
                at = [at[0][h * rep:(h + 1) * rep].contiguous(), at[1][h:h + 1].contiguous(), at[2][h:h + 1].contiguous()]
                if back:
                    at = [t.requires_grad_() for t in at]
                out, lse = _attention64(*at, rep)
                if back:
                    do = s["do"][t0:t0 + n].double().transpose(0, 1)[h * rep:(h + 1) * rep].contiguous()
                    got = torch.autograd.grad(out, at, do)
                else:
                    got = (out, lse)
                for x, t in zip(names, got):
                    parts[x].append(t)
            for x in names:
                found[x].append(torch.cat(parts[x]).transpose(0, 1))
        found = {x: torch.cat(t) for x, t in found.items()}
        if not back and not case["lse"]:
            del found["lse"]
        return found
    if op in ("norm", "norm_backward"):
        back = op == "norm_backward"
        leaf = lambda t: None if t is None else t.double().requires_grad_(back)  # noqa: E731
        r, b, gamma, post, gate = (leaf(s[x]) for x in ("r", "b", "gamma", "post", "gate"))
        norm = lambda x, w: x * torch.rsqrt(x.pow(2).mean(1, keepdim=True) + EPS) * w  # noqa: E731

        def added():
            t = b if post is None else norm(b, post)
            return case["alpha"] * (t if gate is None else t * gate)

        if not back:
            h = r if b is None else r + added()
            y = norm(h, gamma)
            return {"y": y} if b is None else {"h": h, "y": y}
        # r is the stream that the norm read; what reaches it goes on into the branch
        dr, dgamma = torch.autograd.grad(norm(r, gamma), (r, gamma), s["dy"].double())
        dr = dr + s["dh"].double()
        out = {"dr": dr, "dgamma": dgamma}
        if b is not None:
            wanted = [(x, t) for x, t in (("db", b), ("dpost", post), ("dgate", gate)) if t is not None]
            for (x, _), t in zip(wanted, torch.autograd.grad(added(), [t for _, t in wanted], dr)):
                out[x] = t
        return out
    if op in ("adapters", "adapters_backward"):
        x, a, b = s["x"].double(), s["a"].double(), s["b"].double()
        which, scale = s["adapter"].tolist(), s["scale"].double()
        low = torch.zeros((s["tokens"], case["rank"]), dtype=torch.float64, device=DEV)
        out, da, db = s["r"].double(), torch.zeros_like(a), torch.zeros_like(b)
        for i, t0 in enumerate(s["q_start"].tolist()[:-1]):
            e, t1 = which[i], t0 + s["lens"][i]
            if e < 0:
                continue
            if op == "adapters":
                low[t0:t1] = torch.mm(x[t0:t1], a[e].t())
                out[t0:t1] += scale[e] * torch.mm(low[t0:t1], b[e].t())
            else:
                dy = s["dy"][t0:t1].double() * scale[e]
                ds = torch.mm(dy, b[e])
                out[t0:t1] += torch.mm(ds, a[e])
                da[e] += torch.mm(ds.t(), x[t0:t1])
                db[e] += torch.mm(dy.t(), s["s"][t0:t1].double())
        if op == "adapters":
            return {"y": out, "s": low} if case["keep"] else {"y": out}
        return {"dx": out, "da": da, "db": db}
    # column by column of the packed words; the weight's rounding to 16 bits is part of the definition
    w, dt = s["w"], DTYPES[case["dtype"]]
    d_out, words = w["packed"].shape
    G = 8 * words if w["group"] == -1 else w["group"]
    full = torch.empty((d_out, 8 * words), dtype=torch.float64, device=DEV)
    for k in range(8):
        full[:, k::8] = ((w["packed"] >> (4 * k)) & 15).double()
    for n, c in enumerate(range(0, 8 * words, G)):
        full[:, c:c + G] = (full[:, c:c + G] - w["zeros"][:, n:n + 1].double()) * w["scales"][:, n:n + 1].double()
    dx = torch.mm(s["dy"].double(), full.float().to(dt).double())
    if s["perm"] is not None:
        dx = dx.index_select(1, torch.argsort(s["perm"].long()))
    return dx if s["r"] is None else dx + s["r"].double()
