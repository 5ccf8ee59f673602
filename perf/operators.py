"""Measured cases of the operators that complete a fine-tuning step: the rotation of queries and
keys, causal attention over packed sequences with its gradient, and the adapters' orthogonalised
update.  run() computes them in plain torch or, with `own` set, through the framework."""
import math

import torch

own = False

# Newton-Schulz coefficients of the orthogonalised update (the Muon optimiser's quintic).
NS_A, NS_B, NS_C, NS_STEPS, NS_EPS = 3.4445, -4.7750, 2.0315, 5, 1e-7


# ------------------------------------------------------------------------------- cases
def listed():
    rope, fwd, bwd, muon = "rope", "attention_fwd", "attention_bwd", "muon"
    return [
        # a short prompt: one launch, where latency counts
        {"name": "rope 64 tokens", "op": rope, "M": 64, "heads": 40, "D": 64, "theta": 5e5, "span": 64,
         "inverse": False, "padded": 0},
        # q|k of a packed batch with rows of padding behind it, far positions, the gradient's direction
        {"name": "rope grad 2047 tokens", "op": rope, "M": 2047, "heads": 14, "D": 128, "theta": 1e6,
         "span": 131072, "inverse": True, "padded": 31},
        # q|k of the largest training batch (4 x 2048 tokens, 24 query and 8 key heads)
        {"name": "rope 8192 tokens", "op": rope, "M": 8192, "heads": 32, "D": 128, "theta": 5e5, "span": 2048,
         "inverse": False, "padded": 0},
        # a few short sequences, one of a single token and one empty: the smallest call
        {"name": "fwd short", "op": fwd, "lens": "1,77,0,50", "hq": 12, "hkv": 2, "D": 128, "padded": 5},
        # the 2048-token batch, 4 x 512, heads of 64
        {"name": "fwd 4x512 d64", "op": fwd, "lens": "512,512,512,512", "hq": 32, "hkv": 8, "D": 64, "padded": 0},
        # documents of uneven length packed to a fixed row count
        {"name": "fwd ragged", "op": fwd, "lens": "2900,17,1023,640,1,129,2051,1300", "hq": 12, "hkv": 2, "D": 128,
         "padded": 131},
        # the largest training batch
        {"name": "fwd 4x2048 d128", "op": fwd, "lens": "2048,2048,2048,2048", "hq": 24, "hkv": 8, "D": 128,
         "padded": 0},
        # the gradients of the same kinds of batch
        {"name": "bwd short", "op": bwd, "lens": "1,77,0,50", "hq": 12, "hkv": 2, "D": 128, "padded": 5},
        {"name": "bwd 1999 d64", "op": bwd, "lens": "700,1,1298", "hq": 32, "hkv": 8, "D": 64, "padded": 0},
        {"name": "bwd 4x2048 d128", "op": bwd, "lens": "2048,2048,2048,2048", "hq": 24, "hkv": 8, "D": 128,
         "padded": 0},
        # the 14 adapter matrices of one layer (rank 16), gradients in BF16
        {"name": "muon one layer", "op": muon, "layers": 1, "r": 16, "H": 2048, "KV": 512, "I": 8192, "fp32": False},
        # the adapters of a whole model of 28 layers, gradients in FP32 as summed over replicas
        {"name": "muon 28 layers", "op": muon, "layers": 28, "r": 16, "H": 1536, "KV": 256, "I": 8960, "fp32": True},
    ]


def _spread(rng, lo, hi):
    """A whole number of [lo, hi], even over its logarithm."""
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _lengths(rng, parts, rows):
    """The lengths of `parts` packed sequences that add up to `rows`, some of them short or empty."""
    cuts = sorted(rng.randint(0, rows) for _ in range(parts - 1))
    return ",".join(str(b - a) for a, b in zip([0] + cuts, cuts + [rows]))


def draw(rng):
    op = rng.choice(["rope", "attention_fwd", "attention_bwd", "muon"])
    if op == "rope":
        D = rng.choice([64, 128])
        M = _spread(rng, 1, 8192)
        return {"op": op, "M": M, "heads": rng.randint(2, 4096 // D), "D": D, "theta": rng.choice([1e4, 5e5, 1e6]),
                "span": rng.choice([64, 4096, 131072]), "inverse": rng.random() < 0.5,
                "padded": rng.choice([0, min(7, M - 1)])}
    if op == "muon":
        r = rng.choice([16, 16, 32, 48])
        return {"op": op, "layers": _spread(rng, 1, 16 if r == 16 else 4), "r": r, "H": _spread(rng, 64, 2048),
                "KV": _spread(rng, 64, 512), "I": _spread(rng, 256, 8192), "fp32": rng.random() < 0.5}
    D = rng.choice([64, 128])
    hkv = rng.choice([1, 2, 4, 8])
    hq = hkv * rng.randint(1, 24 // hkv if D == 128 else 32 // hkv)
    parts = rng.randint(1, 8)
    rows = _spread(rng, 1, int(4096 / parts ** 0.5))
    return {"op": op, "lens": _lengths(rng, parts, rows), "hq": hq, "hkv": hkv, "D": D, "padded": rng.choice([0, 3, 130])}


# ------------------------------------------------------------------------------ inputs
def _normal(g, *shape, std=1.0, dtype=torch.bfloat16):
    return (torch.randn(shape, generator=g, device="cuda", dtype=torch.float32) * std).to(dtype)


def _starts(lens):
    out = [0]
    for n in lens:
        out.append(out[-1] + n)
    return out


def _muon_groups(case):
    """(matrices, rows, columns) of the adapters by shape: A [r x in] and B [out x r] of q, k, v, o,
    gate, up and down."""
    L, r, H, KV, I = (case[k] for k in ("layers", "r", "H", "KV", "I"))
    return [(6 * L, r, H), (L, r, I), (3 * L, H, r), (2 * L, KV, r), (2 * L, I, r)]


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    op = case["op"]
    if op == "rope":
        M, heads, D = case["M"], case["heads"], case["D"]
        pos = torch.randint(0, case["span"], (M,), generator=g, device="cuda", dtype=torch.int32)
        if case["padded"]:
            pos[M - case["padded"]:] = -1          # rows behind the last sequence
        # q|k are the leading columns of wider rows (v follows), as a fused projection writes them
        x = _normal(g, M, heads * D + 2 * D)
        inv_freq = case["theta"] ** (-torch.arange(0, D, 2, dtype=torch.float64) / D)
        return {"op": op, "x": x[:, :heads * D], "y": torch.zeros((M, heads * D), dtype=x.dtype, device="cuda"),
                "pos": pos, "inv_freq": inv_freq, "heads": heads, "D": D, "inverse": case["inverse"]}
    if op == "muon":
        gdt = torch.float32 if case["fp32"] else torch.bfloat16
        groups = []
        for n, rows, cols in _muon_groups(case):
            # gradients of unequal directions (a few strong ones), as an adapter's are
            r = min(rows, cols)
            mix = torch.exp(_normal(g, n, r, r, dtype=torch.float32)) * _normal(g, n, r, r, dtype=torch.float32)
            raw = lambda: _normal(g, n, rows, cols, std=1e-3, dtype=torch.float32)  # noqa: E731
            shaped = (lambda t: mix @ t) if rows <= cols else (lambda t: t @ mix)
            w = _normal(g, n, rows, cols, std=0.02, dtype=torch.float32)
            groups.append({"g": shaped(raw()).to(gdt), "m": shaped(raw()), "w": w, "m_out": torch.zeros_like(w),
                           "w_out": torch.zeros_like(w), "w16": torch.zeros_like(w, dtype=torch.bfloat16)})
        return {"op": op, "groups": groups, "lr": 0.02, "momentum": 0.95, "weight_decay": 0.01}
    lens = [int(n) for n in case["lens"].split(",")]
    hq, hkv, D = case["hq"], case["hkv"], case["D"]
    starts = _starts(lens)
    M = starts[-1] + case["padded"]
    qkv = _normal(g, M, (hq + 2 * hkv) * D)
    bf = lambda *sh: torch.zeros(sh, dtype=torch.bfloat16, device="cuda")  # noqa: E731
    st = {"op": op, "q": qkv[:, :hq * D], "k": qkv[:, hq * D:(hq + hkv) * D], "v": qkv[:, (hq + hkv) * D:],
          "cu": torch.tensor(starts, dtype=torch.int32, device="cuda"), "hq": hq, "hkv": hkv, "D": D,
          "longest": max(lens)}
    if op == "attention_fwd":
        return st | {"o": bf(M, hq * D), "lse": torch.zeros((hq, M), dtype=torch.float32, device="cuda")}
    o, lse = _plain_fwd(st)          # what the forward pass left for its gradient
    dqkv = bf(M, (hq + 2 * hkv) * D)
    return st | {"o": o, "lse": lse, "do": _normal(g, M, hq * D), "dq": dqkv[:, :hq * D],
                 "dk": dqkv[:, hq * D:(hq + hkv) * D], "dv": dqkv[:, (hq + hkv) * D:]}


# ------------------------------------------------------------------------ plain forms
def _plain_rope(st):
    M, heads, D = st["x"].shape[0], st["heads"], st["D"]
    ang = st["pos"].double()[:, None] * st["inv_freq"].cuda()[None, :]      # far positions need 64 bits
    c, s = torch.cos(ang).float()[:, None, :], torch.sin(ang).float()[:, None, :]
    if st["inverse"]:
        s = -s
    x = st["x"].float().reshape(M, heads, D)
    a, b = x[..., :D // 2], x[..., D // 2:]
    y = torch.cat([a * c - b * s, b * c + a * s], -1).reshape(M, heads * D)
    return torch.where((st["pos"] >= 0)[:, None], y, 0.0).to(torch.bfloat16)


def _padded(st):
    """Row numbers [sequences x longest] of the packed batch and which of them exist."""
    cu = st["cu"].long()
    n = torch.arange(st["longest"], device="cuda")
    live = n[None, :] < (cu[1:] - cu[:-1])[:, None]
    return torch.where(live, cu[:-1, None] + n[None, :], 0), live


def _heads(t, rows, live, heads, D, group=1):
    """[sequences x heads x longest x D] in 32 bits, each head repeated for its group, dead rows zero."""
    x = torch.where(live[..., None], t[rows].float(), 0.0).reshape(*rows.shape, heads, D).transpose(1, 2)
    return x.repeat_interleave(group, 1)


def _packed(x, rows, live, M):
    """Back to [M x heads D], rows of no sequence zero."""
    out = torch.zeros((M, x.shape[1] * x.shape[3]), dtype=torch.float32, device="cuda")
    out[rows[live]] = x.transpose(1, 2).flatten(2)[live]
    return out


def _probabilities(st, rows, live):
    """exp(scores - their row's log-sum) over the keys a row may see, and the log-sums."""
    hq, hkv, D = st["hq"], st["hkv"], st["D"]
    q = _heads(st["q"], rows, live, hq, D)
    k = _heads(st["k"], rows, live, hkv, D, hq // hkv)
    s = q @ k.transpose(-1, -2) * D ** -0.5
    n = torch.arange(s.shape[-1], device="cuda")
    s = s.masked_fill(n[None, :] > n[:, None], float("-inf"))
    top = s.amax(-1, keepdim=True)
    p = torch.exp(s - top)
    total = p.sum(-1, keepdim=True)
    return q, k, p / total, (top + torch.log(total))[..., 0]


def _plain_fwd(st):
    hq, hkv, D, M = st["hq"], st["hkv"], st["D"], st["q"].shape[0]
    rows, live = _padded(st)
    _, _, p, logs = _probabilities(st, rows, live)
    o = p @ _heads(st["v"], rows, live, hkv, D, hq // hkv)
    lse = torch.zeros((hq, M), dtype=torch.float32, device="cuda")
    lse[:, rows[live]] = logs.transpose(0, 1)[:, live]
    return _packed(o, rows, live, M).to(torch.bfloat16), lse


def _plain_bwd(st):
    hq, hkv, D, M = st["hq"], st["hkv"], st["D"], st["q"].shape[0]
    rows, live = _padded(st)
    q, k, p, _ = _probabilities(st, rows, live)
    v = _heads(st["v"], rows, live, hkv, D, hq // hkv)
    do = _heads(st["do"], rows, live, hq, D)
    delta = (do * _heads(st["o"], rows, live, hq, D)).sum(-1, keepdim=True)
    grouped = lambda t: t.reshape(t.shape[0], hkv, hq // hkv, *t.shape[2:]).sum(2)  # noqa: E731
    dv = grouped(p.transpose(-1, -2) @ do)
    ds = p * (do @ v.transpose(-1, -2) - delta) * D ** -0.5
    dk = grouped(ds.transpose(-1, -2) @ q)
    return tuple(_packed(t, rows, live, M).to(torch.bfloat16) for t in (ds @ k, dk, dv))


def _orthogonal(u):
    """Newton-Schulz products of a batch of matrices, on the side of their few rows or columns."""
    tall = u.shape[-2] > u.shape[-1]
    x = u.transpose(-1, -2) if tall else u
    x = x / (x.square().sum((-1, -2), keepdim=True).sqrt() + NS_EPS)
    for _ in range(NS_STEPS):
        a = x @ x.transpose(-1, -2)
        x = NS_A * x + (NS_B * a + NS_C * (a @ a)) @ x
    return x.transpose(-1, -2) if tall else x


def _muon_group(gr, lr, mu, wd):
    grad = gr["g"].float()
    m = mu * gr["m"] + grad
    rows, cols = m.shape[-2:]
    w = (1 - lr * wd) * gr["w"] - lr * math.sqrt(max(1.0, rows / cols)) * _orthogonal(grad + mu * m)
    return m, w, w.to(torch.bfloat16)


def _plain_muon(st):
    return [_muon_group(gr, st["lr"], st["momentum"], st["weight_decay"]) for gr in st["groups"]]


def run(state):
    op = state["op"]
    if not own:
        plain = {"rope": _plain_rope, "attention_fwd": _plain_fwd, "attention_bwd": _plain_bwd, "muon": _plain_muon}
        return plain[op](state)
    import nvfp4_gemm_b200 as P
    st = state
    if op == "rope":
        return P.pact_rope(st["x"], st["pos"], st["inv_freq"], st["heads"], y=st["y"], inverse=st["inverse"])
    if op == "attention_fwd":
        return P.pact_attention_fwd(st["q"], st["k"], st["v"], st["cu"], st["hq"], st["hkv"], o=st["o"],
                                    lse=st["lse"])
    if op == "attention_bwd":
        return P.pact_attention_bwd(st["do"], st["q"], st["k"], st["v"], st["o"], st["lse"], st["cu"], st["hq"],
                                    st["hkv"], dq=st["dq"], dk=st["dk"], dv=st["dv"])
    col = lambda key: [gr[key] for gr in st["groups"]]  # noqa: E731
    P.pact_muon_step(col("w"), col("g"), col("m"), lr=st["lr"], momentum=st["momentum"],
                     weight_decay=st["weight_decay"], weights_out=col("w_out"), momenta_out=col("m_out"),
                     weights_bf16=col("w16"))
    return [(gr["m_out"], gr["w_out"], gr["w16"]) for gr in st["groups"]]


# -------------------------------------------------------------------------------- work
def work(case):
    op = case["op"]
    if op == "rope":
        live = case["M"] - case["padded"]
        return {"bytes": 4 * live * case["heads"] * case["D"] + 4 * case["M"],
                "flops": 3 * live * case["heads"] * case["D"]}
    if op == "muon":
        r = case["r"]
        n = sum(c * rows * cols for c, rows, cols in _muon_groups(case))
        # in: gradient, momentum, weight; out: momentum, weight, its BF16 copy
        return {"bytes": n * ((4 if case["fp32"] else 2) + 4 + 4 + 4 + 4 + 2), "flops": 4 * n * r}
    lens = [int(n) for n in case["lens"].split(",")]
    hq, hkv, D, rows = case["hq"], case["hkv"], case["D"], sum(lens)
    pairs = hq * sum(n * (n + 1) // 2 for n in lens)
    if op == "attention_fwd":
        return {"bytes": 2 * rows * D * (2 * hq + 2 * hkv) + 4 * rows * hq, "flops": 4 * D * pairs}
    return {"bytes": 2 * rows * D * (4 * hq + 4 * hkv) + 4 * rows * hq, "flops": 10 * D * pairs}


# ------------------------------------------------------------------------- in 64 bits
def exact(case, seed):
    st = prepare(case, seed)
    op = case["op"]
    if op == "rope":
        D, heads = case["D"], case["heads"]
        x = st["x"].double().reshape(-1, heads, 2, D // 2)
        turn = torch.polar(torch.ones((), dtype=torch.float64, device="cuda"),
                           st["pos"].double()[:, None] * st["inv_freq"].cuda())
        z = torch.complex(x[:, :, 0], x[:, :, 1]) * (turn.conj() if case["inverse"] else turn)[:, None]
        y = torch.stack([z.real, z.imag], 2).reshape(-1, heads * D)
        y[st["pos"] < 0] = 0
        return y
    if op == "muon":
        out = []
        for gr in st["groups"]:
            m = gr["m"].double() * st["momentum"] + gr["g"].double()
            u = gr["g"].double() + st["momentum"] * m
            rows, cols = m.shape[-2:]
            gram = u.mT @ u if rows > cols else u @ u.mT
            square, axes = torch.linalg.eigh(gram)
            square = square.clamp_min(0)
            # the products scale each direction of u by a polynomial of its singular value
            sigma = square.sqrt() / (square.sum(-1, keepdim=True).sqrt() + NS_EPS)
            gain = 1 / (square.sum(-1, keepdim=True).sqrt() + NS_EPS)
            for _ in range(NS_STEPS):
                f = NS_A + NS_B * sigma ** 2 + NS_C * sigma ** 4
                sigma, gain = sigma * f, gain * f
            p = (axes * gain[..., None, :]) @ axes.mT
            turned = u @ p if rows > cols else p @ u
            w = gr["w"].double() * (1 - st["lr"] * st["weight_decay"])
            w = w - st["lr"] * max(1.0, rows / cols) ** 0.5 * turned
            out.append((m, w, w))
        return out
    lens = [int(n) for n in case["lens"].split(",")]
    hq, hkv, D = case["hq"], case["hkv"], case["D"]
    M = st["q"].shape[0]
    heads = lambda t, n: t.double().reshape(M, n, D)  # noqa: E731
    q, k, v = heads(st["q"], hq), heads(st["k"], hkv), heads(st["v"], hkv)
    o = torch.zeros((M, hq, D), dtype=torch.float64, device="cuda")
    lse = torch.zeros((hq, M), dtype=torch.float64, device="cuda")
    dq, dk, dv = torch.zeros_like(o), torch.zeros_like(k), torch.zeros_like(v)
    for a, b in zip(_starts(lens), _starts(lens)[1:]):
        if a == b:
            continue
        hide = torch.ones((b - a, b - a), dtype=torch.bool, device="cuda").triu(1)
        for h in range(hq):
            g = h // (hq // hkv)
            s = ((q[a:b, h] @ k[a:b, g].T) / math.sqrt(D)).masked_fill_(hide, -math.inf)
            lse[h, a:b] = torch.logsumexp(s, -1)
            p = torch.exp(s - lse[h, a:b, None])
            o[a:b, h] = p @ v[a:b, g]
            if op == "attention_bwd":
                do = st["do"][a:b].double().reshape(b - a, hq, D)[:, h]
                dp = do @ v[a:b, g].T
                ds = p * (dp - (dp * p).sum(-1, keepdim=True)) / math.sqrt(D)
                dv[a:b, g] += p.T @ do
                dq[a:b, h] = ds @ k[a:b, g]
                dk[a:b, g] += ds.T @ q[a:b, h]
    if op == "attention_fwd":
        return o.reshape(M, -1), lse
    return dq.reshape(M, -1), dk.reshape(M, -1), dv.reshape(M, -1)
