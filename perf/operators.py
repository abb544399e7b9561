"""Cases of the operators around the TTT layer: rotary positions with several axes,
the gated linear recurrence, and group norm with an activation.

A case names its operator ("rope", "scan" or "norm"), its sizes and its options.
`run` computes one pass in elementary torch operations, or, where `own` is true,
through this repository's package.  `exact` evaluates the same definitions in
64 bits, by other means.
"""
import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


# --------------------------------------------------------------------- cases
def _rope(name, B, H, N, grid, pairs, d, base, pairing, dtype, tokens_first, backward):
    return {"name": name, "op": "rope", "B": B, "H": H, "N": N, "grid": grid, "pairs": pairs, "d": d, "base": base,
            "pairing": pairing, "dtype": dtype, "tokens_first": tokens_first, "backward": backward}


def _scan(name, B, L, D, gate, inp, dtype, train, ragged, packed, state):
    return {"name": name, "op": "scan", "B": B, "L": L, "D": D, "gate": gate, "inp": inp, "dtype": dtype,
            "train": train, "ragged": ragged, "packed": packed, "state": state}


def _norm(name, B, N, C, G, act, dtype, train, heads_first):
    return {"name": name, "op": "norm", "B": B, "N": N, "C": C, "G": G, "act": act, "dtype": dtype, "train": train,
            "heads_first": heads_first}


def listed():
    return [
        # one new token of each of eight sequences (a streamed layer's query): latency counts
        _rope("rope_one_token", 8, 6, 1, "1x1", "16,16", 64, 100.0, "halves", "bf16", False, False),
        # the queries of a 78 x 78 patch grid, read out of the projection's [B, N, H, d], written heads first
        _rope("rope_vit_78x78", 8, 6, 6084, "78x78", "16,16", 64, 100.0, "halves", "bf16", True, False),
        # the keys of 48 views of 64 x 64 patches, time, height and width, a quarter of each head left unrotated
        _rope("rope_views_196k", 1, 2, 196608, "48x64x64", "32,80,80", 512, 10000.0, "interleaved", "bf16", True,
              False),
        # the gradient of a small fp32 video clip's keys, an odd grid and a head that is not a power of two
        _rope("rope_clip_grad_f32", 2, 5, 2583, "7x9x41", "8,12,12", 80, 10000.0, "halves", "f32", False, True),
        # one new token of each sequence, the state carried from call to call: latency counts
        _scan("scan_one_token", 8, 1, 384, "sigmoid", "complement", "bf16", False, False, False, True),
        # a training step of the causal language layer's width and length, gate and input out of one projection
        _scan("scan_lm_train_32k", 2, 32768, 1024, "sigmoid", "complement", "bf16", True, False, True, False),
        # one forward pass over a million tokens of a scene
        _scan("scan_scene_1m", 1, 1029120, 1024, "exp", "plain", "bf16", False, False, False, True),
        # a padded fp32 batch of odd lengths and an odd width, with its gradients
        _scan("scan_ragged_train_f32", 5, 5001, 333, "value", "plain", "f32", True, True, False, True),
        # a small image's tokens: latency counts
        _norm("norm_196", 1, 196, 64, 8, "silu", "bf16", False, False),
        # the layer's output [B, H, N, d], one group a head, written tokens first
        _norm("norm_heads_78x78", 8, 6084, 384, 6, "silu", "bf16", False, True),
        # a training step on the full-size feature map of an image decoder
        _norm("norm_image_train_1024", 2, 1048576, 128, 32, "silu", "bf16", True, False),
        # odd sizes in fp32 with the gradients, three channels a group
        _norm("norm_odd_train_f32", 3, 1001, 96, 32, "gelu", "f32", True, False),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["rope", "scan", "norm"])
    dtype = rng.choice(["bf16", "bf16", "f32"])
    if op == "rope":
        axes = rng.choice([1, 2, 3])
        sides = [_log(rng, 1, {1: 200000, 2: 300, 3: 56}[axes]) for _ in range(axes)]
        pairs = [rng.choice([4, 7, 8, 11, 16, 32, 40]) for _ in range(axes)]
        N = math.prod(sides)
        d = 2 * sum(pairs) + rng.choice([0, 0, 0, 2, 16])
        H = rng.choice([1, 2, 3, 4, 6, 12, 16])
        B = max(1, min(rng.choice([1, 2, 3, 8]), 200_000_000 // (N * H * d)))
        H = max(1, min(H, 200_000_000 // (N * B * d)))
        case = _rope("", B, H, N, "x".join(map(str, sides)), ",".join(map(str, pairs)), d,
                     rng.choice([100.0, 10000.0, 500000.0]), rng.choice(["halves", "interleaved"]), dtype,
                     rng.random() < 0.5, rng.random() < 0.5)
    elif op == "scan":
        L = _log(rng, 1, 500000)
        D = _log(rng, 1, 4096)
        if rng.random() < 0.6:
            D = max(8, D // 8 * 8)
        B = max(1, min(rng.choice([1, 2, 3, 5, 8, 16]), 200_000_000 // (L * D)))
        D = max(1, min(D, 200_000_000 // (L * B)))
        case = _scan("", B, L, D, rng.choice(["value", "sigmoid", "exp"]), rng.choice(["plain", "complement"]), dtype,
                     rng.random() < 0.5, rng.random() < 0.3, rng.random() < 0.5, rng.random() < 0.5)
    else:
        N = _log(rng, 1, 600000)
        G = rng.choice([1, 2, 6, 8, 16, 32])
        C = G * _log(rng, 1, max(2, 1024 // G))
        B = max(1, min(rng.choice([1, 2, 3, 8, 16]), 130_000_000 // (N * C)))
        N = max(1, min(N, 130_000_000 // (B * C)))
        # the gradient of one or two values a group is nothing but rounding: training cases have more
        train = rng.random() < 0.5 and N * (C // G) >= 32
        case = _norm("", B, N, C, G, rng.choice(["none", "silu", "gelu"]), dtype, train, rng.random() < 0.3)
    del case["name"]
    return case


def _ints(text, sep=","):
    return [int(t) for t in text.split(sep)]


# ------------------------------------------------------------------- prepare
def _randn(gen, *shape):
    return torch.randn(shape, generator=gen, device="cuda", dtype=torch.float32)


def _lengths(case, seed):
    """Lengths of a padded batch: one full, one empty where there are three or more, the others between."""
    gen = torch.Generator().manual_seed(seed + 17)
    n = torch.randint(1, case["L"] + 1, (case["B"],), generator=gen, dtype=torch.int32)
    n[0] = case["L"]
    if case["B"] > 2:
        n[1] = 0
    return n.cuda()


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    dt = DTYPES[case["dtype"]]
    s = {"case": case}
    if case["op"] == "rope":
        B, H, N, d = case["B"], case["H"], case["N"], case["d"]
        x = _randn(gen, B, N, H, d).to(dt) if case["tokens_first"] else _randn(gen, B, H, N, d).to(dt)
        s["x"] = x.transpose(1, 2) if case["tokens_first"] else x
        # raster positions of the grid, from where an earlier part of the stream ended
        sides = _ints(case["grid"], "x")
        t = torch.arange(N, device="cuda", dtype=torch.int64)
        at = []
        for side in reversed(sides):
            at.append(t % side)
            t = t // side
        at.reverse()
        at[0] = at[0] + seed % 1000
        s["pos"] = torch.stack(at, dim=1).to(torch.int32)
        # the plan of the plain form: the axis and the frequency of every pair
        pairs = _ints(case["pairs"])
        s["axis"] = torch.tensor([k for k, n in enumerate(pairs) for _ in range(n)], device="cuda")
        s["freq"] = torch.tensor([case["base"] ** (-j / n) for n in pairs for j in range(n)], device="cuda",
                                 dtype=torch.float64)
    elif case["op"] == "scan":
        B, L, D = case["B"], case["L"], case["D"]
        if case["packed"]:
            both = torch.empty((B, L, 2 * D), device="cuda", dtype=dt)
            g, x = both[..., :D], both[..., D:]
        else:
            g, x = (torch.empty((B, L, D), device="cuda", dtype=dt) for _ in range(2))
        z = _randn(gen, B, L, D)
        if case["gate"] == "sigmoid":
            g.copy_(z + 2.5)
        elif case["gate"] == "exp":
            g.copy_(-0.2 * torch.nn.functional.softplus(z))
        else:
            g.copy_(1.0 - 0.2 * torch.sigmoid(z))
        del z
        x.copy_(_randn(gen, B, L, D))
        s["g"], s["x"] = g, x
        s["h0"] = _randn(gen, B, D) if case["state"] else None
        s["lengths"] = _lengths(case, seed) if case["ragged"] else None
        if case["train"]:
            s["dh"] = _randn(gen, B, L, D).to(dt)
            s["dh_last"] = _randn(gen, B, D) if case["state"] else None
    else:
        B, N, C, G = case["B"], case["N"], case["C"], case["G"]
        shape = (B, G, N, C // G) if case["heads_first"] else (B, N, C)
        s["x"] = (_randn(gen, *shape) * 1.5 + 0.5).to(dt)
        s["weight"] = 1.0 + 0.2 * _randn(gen, C)
        s["bias"] = 0.2 * _randn(gen, C)
        if case["train"]:
            s["dy"] = _randn(gen, B, N, C).to(dt)
    if own:
        s["op"] = _operator(case)
    return s


# ---------------------------------------------------- this repository's kernels
def _operator(case):
    from weight_sequence_mixing_b200 import token_ops

    if case["op"] == "rope":
        return token_ops.RotaryPositions(dict(d=case["d"], pairs=_ints(case["pairs"]), base=case["base"],
                                              pairing=case["pairing"], dtype=case["dtype"]))
    if case["op"] == "scan":
        return token_ops.GatedScan(dict(D=case["D"], gate=case["gate"], inp=case["inp"], dtype=case["dtype"]))
    return token_ops.GroupNorm(dict(C=case["C"], groups=case["G"], act=case["act"], eps=1e-5, dtype=case["dtype"]))


def _run_own(s):
    case, op = s["case"], s["op"]
    if case["op"] == "rope":
        return op.backward(s["x"], s["pos"]) if case["backward"] else op.forward(s["x"], s["pos"])
    if case["op"] == "scan":
        saved = op.new_saved(case["B"], case["L"]) if case["train"] else None
        h, h_last = op.forward(s["g"], s["x"], h0=s["h0"], lengths=s["lengths"], saved=saved)
        if not case["train"]:
            return {"h": h, "h_last": h_last}
        dg, dx, dh0 = op.backward(s["dh"], s["g"], s["x"], saved, dh_last=s["dh_last"], lengths=s["lengths"])
        return {"h": h, "h_last": h_last, "dg": dg, "dx": dx, "dh0": dh0}
    stats = op.new_stats(case["B"]) if case["train"] else None
    y = op.forward(s["x"], s["weight"], s["bias"], stats=stats)
    if not case["train"]:
        return {"y": y}
    dx, dweight, dbias = op.backward(s["dy"], s["x"], s["weight"], s["bias"], stats)
    return {"y": y, "dx": dx, "dweight": dweight, "dbias": dbias}


# ------------------------------------------------------------------ plain forms
def _plain_rope(s):
    case = s["case"]
    x, pos = s["x"], s["pos"]
    angle = pos.double()[:, s["axis"]] * s["freq"]
    cos, sin = torch.cos(angle).float(), torch.sin(angle).float()
    sin = -sin if case["backward"] else sin
    m = angle.shape[1]
    xf = x.float()
    if case["pairing"] == "halves":
        a, b = xf[..., :m], xf[..., m:2 * m]
        y = torch.cat([a * cos - b * sin, b * cos + a * sin, xf[..., 2 * m:]], dim=-1)
    else:
        a, b = xf[..., 0:2 * m:2], xf[..., 1:2 * m:2]
        y = torch.stack([a * cos - b * sin, b * cos + a * sin], dim=-1).flatten(-2)
        y = torch.cat([y, xf[..., 2 * m:]], dim=-1)
    return y.to(x.dtype)


def _pair_scan(a, u):
    """h_t = a_t h_{t-1} + u_t along dim 1 (h before the first row is zero): neighbouring steps are
    joined into one, the half as long scan gives every second row, and one product fills the others."""
    L = a.shape[1]
    if L == 1:
        return u
    even, odd = slice(0, L - L % 2, 2), slice(1, None, 2)
    S = _pair_scan(a[:, odd] * a[:, even], a[:, odd] * u[:, even] + u[:, odd])
    h = torch.empty_like(u)
    h[:, odd] = S
    h[:, 0] = u[:, 0]
    rest = (L - 1) // 2
    h[:, 2::2] = a[:, 2::2] * S[:, :rest] + u[:, 2::2]
    return h


def _plain_scan(s):
    case = s["case"]
    g, x = s["g"].float(), s["x"].float()
    dt = s["x"].dtype
    B, L, D = x.shape
    if case["gate"] == "sigmoid":
        a, rest = torch.sigmoid(g), torch.sigmoid(-g)
    elif case["gate"] == "exp":
        a, rest = torch.exp(g), -torch.expm1(g)
    else:
        a, rest = g, 1.0 - g
    u = rest * x if case["inp"] == "complement" else x
    keep = None
    if s["lengths"] is not None:
        keep = (torch.arange(L, device=x.device)[None, :] < s["lengths"][:, None])[..., None]
        a, u = torch.where(keep, a, 1.0), torch.where(keep, u, 0.0)
    h0 = s["h0"] if s["h0"] is not None else torch.zeros((B, D), device=x.device)
    h = _pair_scan(a, torch.cat([(u[:, 0] + a[:, 0] * h0)[:, None], u[:, 1:]], dim=1))
    out = {"h": (h if keep is None else torch.where(keep, h, 0.0)).to(dt), "h_last": h[:, -1].clone()}
    if not case["train"]:
        return out
    dh = s["dh"].float()
    if keep is not None:
        dh = torch.where(keep, dh, 0.0)
    last = dh[:, -1] + s["dh_last"] if s["dh_last"] is not None else dh[:, -1]
    after = torch.cat([a[:, 1:], torch.ones_like(a[:, :1])], dim=1)
    lam = _pair_scan(after.flip(1), torch.cat([last[:, None], dh.flip(1)[:, 1:]], dim=1)).flip(1)
    before = torch.cat([h0[:, None], h[:, :-1]], dim=1)
    if case["inp"] == "complement":
        dx, da = rest * lam, lam * (before - x)
    else:
        dx, da = lam, lam * before
    dg = da if case["gate"] == "value" else da * a if case["gate"] == "exp" else da * a * rest
    if keep is not None:
        dg, dx = torch.where(keep, dg, 0.0), torch.where(keep, dx, 0.0)
    return {**out, "dg": dg.to(dt), "dx": dx.to(dt), "dh0": a[:, 0] * lam[:, 0]}


def _by_group(x, case):
    """[B, N, C] or [B, G, N, C/G] as [B, G, N, C/G]."""
    return x if case["heads_first"] else x.unflatten(-1, (case["G"], -1)).transpose(1, 2)


def _plain_norm(s):
    case = s["case"]
    B, N, C, G = case["B"], case["N"], case["C"], case["G"]
    dt = s["x"].dtype
    x = _by_group(s["x"], case).float()
    w, b = s["weight"].view(G, 1, -1), s["bias"].view(G, 1, -1)
    mean = x.mean(dim=(2, 3), keepdim=True)
    xc = x - mean
    rstd = torch.rsqrt((xc * xc).mean(dim=(2, 3), keepdim=True) + 1e-5)
    xhat = xc * rstd
    z = xhat * w + b
    if case["act"] == "silu":
        y = z * torch.sigmoid(z)
    elif case["act"] == "gelu":
        y = 0.5 * z * (1.0 + torch.erf(z * math.sqrt(0.5)))
    else:
        y = z
    out = {"y": y.to(dt).transpose(1, 2).reshape(B, N, C)}
    if not case["train"]:
        return out
    dy = s["dy"].float().view(B, N, G, C // G).transpose(1, 2)
    if case["act"] == "silu":
        sg = torch.sigmoid(z)
        dz = dy * sg * (1.0 + z * (1.0 - sg))
    elif case["act"] == "gelu":
        dz = dy * (0.5 * (1.0 + torch.erf(z * math.sqrt(0.5))) + z * torch.exp(-0.5 * z * z) / math.sqrt(2 * math.pi))
    else:
        dz = dy
    out["dweight"] = (dz * xhat).sum(dim=(0, 2)).reshape(C)
    out["dbias"] = dz.sum(dim=(0, 2)).reshape(C)
    dhat = dz * w
    dx = rstd * (dhat - dhat.mean(dim=(2, 3), keepdim=True) - xhat * (dhat * xhat).mean(dim=(2, 3), keepdim=True))
    dx = dx.to(dt)
    out["dx"] = dx.contiguous() if case["heads_first"] else dx.transpose(1, 2).reshape(B, N, C)
    return out


def run(state):
    if own:
        return _run_own(state)
    return {"rope": _plain_rope, "scan": _plain_scan, "norm": _plain_norm}[state["case"]["op"]](state)


# ------------------------------------------------------------------------ work
def work(case):
    e = 2 if case["dtype"] == "bf16" else 4
    if case["op"] == "rope":
        n = case["B"] * case["H"] * case["N"] * case["d"]
        pairs = _ints(case["pairs"])
        return {"bytes": 2 * n * e + 4 * case["N"] * len(pairs),
                "flops": 6 * case["B"] * case["H"] * case["N"] * sum(pairs)}
    if case["op"] == "scan":
        n, ends = case["B"] * case["L"] * case["D"], 4 * case["B"] * case["D"]
        if case["train"]:  # g, x, dh in; h, dg, dx out
            return {"bytes": 6 * n * e + ends * (2 + 2 * bool(case["state"])), "flops": 20 * n}
        return {"bytes": 3 * n * e + ends * (1 + bool(case["state"])), "flops": 6 * n}
    n, c = case["B"] * case["N"] * case["C"], 4 * case["C"]
    if case["train"]:  # x, dy in; y, dx out
        return {"bytes": 4 * n * e + 4 * c, "flops": 40 * n}
    return {"bytes": 2 * n * e + 2 * c, "flops": 15 * n}


# ------------------------------------------------------------ the definitions in 64 bits
def _exact_rope(case, s):
    x = s["x"].to(torch.float64)
    pairs, m = _ints(case["pairs"]), sum(_ints(case["pairs"]))
    y = x.clone()
    sign = -1.0 if case["backward"] else 1.0
    at = 0
    for axis, n in enumerate(pairs):
        p = s["pos"][:, axis].to(torch.float64)
        for j in range(n):
            turn = p * case["base"] ** (-j / n)
            c, sn = torch.cos(turn), sign * torch.sin(turn)
            i, k = (at, at + m) if case["pairing"] == "halves" else (2 * at, 2 * at + 1)
            y[..., i] = x[..., i] * c - x[..., k] * sn
            y[..., k] = x[..., i] * sn + x[..., k] * c
            at += 1
    return y


def _steps(a, u, h0):
    """h_t = a_t h_{t-1} + u_t for [B, L, D] in 64 bits: the rows of many stretches step by step
    beside one another, then the stretches one after the other."""
    B, L, D = u.shape
    n = max(1, math.isqrt(L))
    S = -(-L // n)
    fill = S * n - L
    a = torch.cat([a, a.new_ones((B, fill, D))], 1).view(B, S, n, D)
    u = torch.cat([u, u.new_zeros((B, fill, D))], 1).view(B, S, n, D)
    h, p = torch.empty_like(u), torch.empty_like(u)
    state, prod = torch.zeros_like(u[:, :, 0]), torch.ones_like(u[:, :, 0])
    for t in range(n):
        state, prod = a[:, :, t] * state + u[:, :, t], prod * a[:, :, t]
        h[:, :, t], p[:, :, t] = state, prod
    carry = h0
    for k in range(S):
        h[:, k] += p[:, k] * carry[:, None]
        carry = h[:, k, -1]
    return h.view(B, S * n, D)[:, :L]


def _exact_scan(case, s):
    parts = []
    for c in range(0, case["D"], 256):
        cols = slice(c, min(c + 256, case["D"]))
        g, x = s["g"][..., cols].double(), s["x"][..., cols].double()
        B, L, D = x.shape
        a = g if case["gate"] == "value" else torch.exp(g) if case["gate"] == "exp" else 1 / (1 + torch.exp(-g))
        u = (1 - a) * x if case["inp"] == "complement" else x
        live = torch.ones((B, L, 1), device=g.device, dtype=torch.bool)
        if s["lengths"] is not None:
            live = (torch.arange(L, device=g.device) < s["lengths"][:, None])[..., None]
        a1, u1 = torch.where(live, a, 1.0), torch.where(live, u, 0.0)
        h0 = s["h0"][:, cols].double() if s["h0"] is not None else a.new_zeros((B, D))
        h = _steps(a1, u1, h0)
        out = {"h": torch.where(live, h, 0.0), "h_last": h[:, -1]}
        if case["train"]:
            dh = torch.where(live, s["dh"][..., cols].double(), 0.0)
            end = s["dh_last"][:, cols].double() if s["dh_last"] is not None else a.new_zeros((B, D))
            # mu_t = a_t (dh_t + mu_{t+1}), the gradient of the state before row t, from the last row on
            mu = _steps(a1.flip(1), (a1 * dh).flip(1), end).flip(1)
            lam = dh + torch.cat([mu[:, 1:], end[:, None]], 1)
            prev = torch.cat([h0[:, None], h[:, :-1]], 1)
            du_dx = 1 - a if case["inp"] == "complement" else torch.ones_like(a)
            dh_da = prev - x if case["inp"] == "complement" else prev
            slope = {"value": torch.ones_like(a), "exp": a, "sigmoid": a * (1 - a)}[case["gate"]]
            out["dg"] = torch.where(live, lam * dh_da * slope, 0.0)
            out["dx"] = torch.where(live, lam * du_dx, 0.0)
            out["dh0"] = mu[:, 0]
        parts.append(out)
    return {k: torch.cat([p[k] for p in parts], -1) for k in parts[0]}


def _exact_norm(case, s):
    B, N, C, G = case["B"], case["N"], case["C"], case["G"]
    n = C // G
    x, y = s["x"], torch.empty((B, N, C), device="cuda", dtype=torch.float64)
    out = {"y": y}
    if case["train"]:
        out["dx"] = torch.empty(x.shape, device="cuda", dtype=torch.float64)
        out["dweight"], out["dbias"] = (torch.zeros(C, device="cuda", dtype=torch.float64) for _ in range(2))
    for b in range(B):
        for k in range(G):
            cols = slice(k * n, (k + 1) * n)
            v = (x[b, k] if case["heads_first"] else x[b, :, cols]).double()
            w, c = s["weight"][cols].double(), s["bias"][cols].double()
            var, mu = torch.var_mean(v, correction=0)
            sd = torch.sqrt(var + 1e-5)
            e = (v - mu) / sd
            z = (e * w + c).requires_grad_(case["train"])
            f = {"none": lambda t: t, "silu": lambda t: t / (1 + torch.exp(-t)),
                 "gelu": lambda t: t * 0.5 * torch.erfc(-t / math.sqrt(2.0))}[case["act"]](z)
            y[b, :, cols] = f.detach()
            if case["train"]:
                dz, = torch.autograd.grad(f, z, s["dy"][b, :, cols].double())
                out["dbias"][cols] += dz.sum(0)
                out["dweight"][cols] += (dz * e).sum(0)
                q = dz * w
                dv = (q - q.mean() - e * (q * e).mean()) / sd
                (out["dx"][b, k] if case["heads_first"] else out["dx"][b, :, cols]).copy_(dv)
    return out


def exact(case, seed):
    s = prepare(case, seed)
    return {"rope": _exact_rope, "scan": _exact_scan, "norm": _exact_norm}[case["op"]](case, s)
