"""The operators of a DSA training step next to the forward: rotary positions, the sparse attention's backward pass, the gradient of the
indexer's objective and the backward pass of the index scores.

Rows [first, first + T) of one causal sequence: row r sits at position first + r, selects n = min(k, first + r + 1) of the positions up to
its own (ascending, padded with -1, as the top-k selection writes them), and keys come from positions 0 .. first + T - 1."""
import math

import torch

own = False

D, D_V, ROPE = 576, 512, 64        # latent width, value width, rotary dims
SCALE = D ** -0.5


# ---------------------------------------------------------------------------------------------------------------- cases
def listed():
    return [
        # one decode step of 64 sequences at ragged positions: the queries' 64 position dims, scaled for long contexts
        dict(name="rope decode 64", op="rope", T=64, H=128, D=64, wide=576, rot=64, off=0, interleaved=True, spread=131072, factor=40.0,
             dtype="bf16", backward=False),
        # the position part of every latent entry of a 128K sequence
        dict(name="rope latent 128K", op="rope", T=131072, H=1, D=64, wide=576, rot=64, off=0, interleaved=True, spread=0, factor=40.0,
             dtype="bf16", backward=False),
        # the indexer queries' gradient on its way back: first half of each head rotated, the rest passed on
        dict(name="rope indexer backward", op="rope", T=5000, H=64, D=128, wide=128, rot=64, off=0, interleaved=False, spread=0, factor=1.0,
             dtype="fp32", backward=True),
        # a short sequence with few heads: launches count
        dict(name="attention backward tiny", op="attn", T=96, first=0, k=128, H=8, blank=0),
        # a ragged piece that starts inside the dense rows, with empty rows of a padded batch
        dict(name="attention backward ragged", op="attn", T=333, first=1700, k=1984, H=128, blank=7),
        # a block of rows of a 32K sequence
        dict(name="attention backward 32K", op="attn", T=2048, first=30720, k=2048, H=128, blank=0),
        # the objective's gradient of a few rows, and of a block of rows of a 32K sequence
        dict(name="objective backward small", op="kl", T=48, first=500, k=320, H=128, blank=0),
        dict(name="objective backward 32K", op="kl", T=2048, first=30720, k=2048, H=128, blank=0),
        # the small indexer, unscaled integers
        dict(name="indexer backward tiny", op="index", T=200, first=0, k=128, heads=4, dim=64, scaled=False, blank=0),
        # a ragged piece with empty rows, and a block of rows of a 32K sequence
        dict(name="indexer backward ragged", op="index", T=777, first=1500, k=1984, heads=64, dim=128, scaled=True, blank=5),
        dict(name="indexer backward 32K", op="index", T=2048, first=30720, k=2048, heads=64, dim=128, scaled=True, blank=0),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["rope", "attn", "attn", "kl", "index"])
    if op == "rope":
        T, H = _log(rng, 1, 16384), rng.choice([1, 1, 3, 8, 16, 64, 128])
        rot = rng.choice([16, 32, 64, 64, 128])
        D = rot + rng.choice([0, 0, 8, 64, 72])
        if T * H > 200000:
            T = 200000 // H + rng.randrange(100)
        return dict(op="rope", T=T, H=H, D=D, wide=max(D, rng.choice([D, D + 8, 576])), rot=rot, off=8 * rng.randrange((D - rot) // 8 + 1),
                    interleaved=rng.random() < 0.5, spread=rng.choice([0, 4096, 131072, 1000000]), factor=rng.choice([1.0, 8.0, 40.0]),
                    dtype=rng.choice(["bf16", "fp32"]), backward=rng.random() < 0.5)
    k = 64 * rng.randrange(2, 33)
    first = rng.choice([0, _log(rng, 1, 28000)])
    blank = rng.choice([0, 0, 3, 11])
    if op == "index":
        heads = rng.choice([4, 64, 64])
        return dict(op=op, T=_log(rng, 1, 2000), first=first, k=k, heads=heads, dim=64 if heads == 4 else 128, scaled=rng.random() < 0.7,
                    blank=blank)
    return dict(op=op, T=_log(rng, 1, 2000), first=first, k=k, H=rng.choice([1, 8, 16, 37, 64, 96, 128, 128, 128]), blank=blank)


# --------------------------------------------------------------------------------------------------------------- inputs
def _normal(g, *shape, dtype=torch.float32):
    return torch.randn(*shape, generator=g, device="cuda").to(dtype)


def _frequencies(rot, factor):
    """Rotation per position of each pair: 10000^(-2i/rot); with a factor, pairs that turn less than once over 4096 positions are slowed
    by it, pairs that turn more than 32 times are kept, those between are blended."""
    i = torch.arange(rot // 2, dtype=torch.float64)
    f = 10000.0 ** (-2.0 * i / rot)
    if factor == 1.0:
        return f, 1.0
    at = [rot * math.log(4096 / (turns * 2 * math.pi)) / (2 * math.log(10000.0)) for turns in (32.0, 1.0)]
    low, high = max(0, math.floor(at[0])), min(rot // 2 - 1, math.ceil(at[1]))
    ramp = ((i - low) / max(high - low, 1e-3)).clamp(0, 1)
    return f / factor * ramp + f * (1 - ramp), 0.1 * math.log(factor) + 1.0


def _selection(g, case):
    """[T, k] selected positions: n distinct ones spread over the row's own past, ascending, then -1; every blank-th row is empty."""
    T, k = case["T"], case["k"]
    m = case["first"] + 1 + torch.arange(T, device="cuda")[:, None]
    n = m.clamp(max=k)
    i = torch.arange(k, device="cuda")[None, :]
    lo, hi = i * m // n, (i + 1) * m // n
    u = torch.rand(T, k, generator=g, device="cuda", dtype=torch.float64)
    idx = torch.where(i < n, lo + (u * (hi - lo)).long(), -1)
    if case["blank"]:
        idx[:: case["blank"]] = -1
    return idx.to(torch.int32)


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    s = dict(case=dict(case))
    T = case["T"]
    if case["op"] == "rope":
        dt = torch.bfloat16 if case["dtype"] == "bf16" else torch.float32
        wide, at = case["wide"], case["wide"] - case["D"]        # the heads are the last D dims of wider rows
        s["x"] = _normal(g, T, case["H"], wide, dtype=dt)[..., at:]
        s["out"] = torch.zeros(T, case["H"], wide, device="cuda", dtype=dt)[..., at:]
        if case["spread"]:
            s["pos"] = torch.randint(0, case["spread"], (T,), generator=g, device="cuda", dtype=torch.int32)
        else:
            s["pos"] = torch.arange(T, device="cuda", dtype=torch.int32)
        f, s["mscale"] = _frequencies(case["rot"], case["factor"])
        s["freq"] = f.cuda()
        return s
    S = case["first"] + T
    s["idx"] = _selection(g, case)
    if case["op"] == "index":
        hi, di = case["heads"], case["dim"]
        if case["scaled"]:
            q, k = _normal(g, T, hi, di), _normal(g, S, di)
            s["q_scale"], s["k_scale"] = q.abs().amax((1, 2)) / 448, k.abs().amax(1) / 448
            q, k = q / s["q_scale"][:, None, None], k / s["k_scale"][:, None]
            s["w"] = _normal(g, T, hi) * hi ** -0.5
        else:
            q = torch.randint(-7, 8, (T, hi, di), generator=g, device="cuda").float()
            k = torch.randint(-7, 8, (S, di), generator=g, device="cuda").float()
            s["q_scale"] = s["k_scale"] = None
            s["w"] = torch.randint(-3, 4, (T, hi), generator=g, device="cuda").float()
        s["q_idx"], s["k_idx"] = q.clamp(-448, 448).to(torch.float8_e4m3fn), k.clamp(-448, 448).to(torch.float8_e4m3fn)
        # the objective's gradient: the difference of two distributions over the selection
        a, b = (_normal(g, T, case["k"]).masked_fill(s["idx"] < 0, -1e30).softmax(1) for _ in range(2))
        s["dsel"] = torch.where(s["idx"] >= 0, a - b, 0.0)
        return s
    H = case["H"]
    s["q"], s["c"] = _normal(g, T, H, D, dtype=torch.bfloat16), _normal(g, S, D, dtype=torch.bfloat16)
    s["lse"] = torch.empty(T, H, device="cuda")
    if case["op"] == "attn":
        s["out"] = torch.empty(T, H, D_V, device="cuda", dtype=torch.bfloat16)
        s["dout"] = _normal(g, T, H, D_V, dtype=torch.bfloat16)
    else:
        s["sel"] = 2 * _normal(g, T, case["k"])
        s["dkl"] = _normal(g, T).abs() / T
    for a in range(0, T, 256):                                   # what the forward pass left: out and lse
        ids = s["idx"][a:a + 256]
        rows = s["c"][ids.clamp(min=0).long()].float()
        x = (s["q"][a:a + 256].float() @ rows.transpose(1, 2)) * SCALE
        x = torch.where((ids >= 0)[:, None], x, -math.inf)
        lse = torch.logsumexp(x, 2)
        s["lse"][a:a + 256] = lse
        if case["op"] == "attn":
            p = torch.where((ids >= 0)[:, None], (x - lse[..., None]).exp(), 0.0)
            s["out"][a:a + 256] = (p @ rows[..., :D_V]).to(torch.bfloat16)
    return s


# ----------------------------------------------------------------------------------------------------------- plain forms
def _rope(s):
    c, x = s["case"], s["x"]
    r, off = c["rot"], c["off"]
    theta = s["pos"].double()[:, None] * s["freq"][None, :]
    cos, sin = (s["mscale"] * theta.cos()).float()[:, None], (s["mscale"] * theta.sin()).float()[:, None]
    if c["backward"]:
        sin = -sin
    part = x[..., off:off + r].float()
    a, b = (part[..., 0::2], part[..., 1::2]) if c["interleaved"] else (part[..., :r // 2], part[..., r // 2:])
    pair = [a * cos - b * sin, a * sin + b * cos]
    turned = torch.stack(pair, -1).flatten(-2) if c["interleaved"] else torch.cat(pair, -1)
    s["out"].copy_(x)
    s["out"][..., off:off + r] = turned.to(x.dtype)
    return s["out"]


def _probabilities(s):
    """(valid [T, 1, k], the selected rows [T, k, 576], P [T, H, k])"""
    on = (s["idx"] >= 0)[:, None]
    rows = s["c"][s["idx"].clamp(min=0).long()].float()
    x = torch.matmul(s["q"].float(), rows.transpose(1, 2)) * SCALE
    return on, rows, torch.where(on, (x - s["lse"][..., None]).exp(), 0.0)


def _attention_backward(s):
    on, rows, p = _probabilities(s)
    dout = s["dout"].float()
    delta = (dout * s["out"].float()).sum(-1, keepdim=True)
    ds = p * (torch.matmul(dout, rows[..., :D_V].transpose(1, 2)) - delta) * SCALE
    dq = torch.matmul(ds, rows)
    del rows
    each = torch.matmul(ds.transpose(1, 2), s["q"].float())
    each[..., :D_V] += torch.matmul(p.transpose(1, 2), dout)
    dc = torch.zeros(s["c"].shape, device="cuda")
    dc.index_add_(0, s["idx"].clamp(min=0).long().flatten(), each.flatten(0, 1))
    return {"dq": dq.to(torch.bfloat16), "dc": dc.to(torch.bfloat16)}


def _objective_backward(s):
    on, _, p = _probabilities(s)
    on = on[:, 0]
    target = p.sum(1)
    target = target / target.sum(1, keepdim=True)
    x = torch.where(on, s["sel"], -math.inf)
    x = (x - x.amax(1, keepdim=True)).exp()
    return torch.where(on, s["dkl"][:, None] * (x / x.sum(1, keepdim=True) - target), 0.0)


def _indexer_backward(s):
    at = s["idx"].clamp(min=0).long()
    q, k = s["q_idx"].float(), s["k_idx"].float()
    dot = torch.matmul(q.double(), k[at].double().transpose(1, 2)).float()        # the sign decides: 64 bits
    if s["case"]["scaled"]:
        q, k = q * s["q_scale"][:, None, None], k * s["k_scale"][:, None]
        dot = dot * s["q_scale"][:, None, None] * s["k_scale"][at][:, None]
    up = torch.where(s["idx"] >= 0, s["dsel"], 0.0)[:, None]
    live = (dot > 0).float() * up
    dw = (dot * live).sum(2)
    live = live * s["w"][..., None]
    dq = torch.matmul(live, k[at])
    dk = torch.zeros_like(k)
    dk.index_add_(0, at.flatten(), torch.matmul(live.transpose(1, 2), q).flatten(0, 1))
    return {"dq": dq.to(torch.bfloat16), "dk": dk.to(torch.bfloat16), "dw": dw}


def run(s):
    op = s["case"]["op"]
    if not own:
        return {"rope": _rope, "attn": _attention_backward, "kl": _objective_backward, "index": _indexer_backward}[op](s)
    import sparse_attention_long_05_b200 as dsa
    if op == "rope":
        call = dsa.dsa_rope_backward if s["case"]["backward"] else dsa.dsa_rope
        return call(s["x"], s["freq"], s["pos"], rot_off=s["case"]["off"], interleaved=s["case"]["interleaved"], mscale=s["mscale"],
                    out=s["out"])
    if op == "attn":
        dq, dc = dsa.dsa_sparse_mla_attn_backward(s["q"], s["c"], s["idx"], s["out"], s["lse"], s["dout"], SCALE)
        return {"dq": dq, "dc": dc}
    if op == "kl":
        return dsa.dsa_indexer_kl_backward(s["q"], s["c"], s["idx"], s["sel"], s["lse"], s["dkl"], SCALE)
    dq, dk, dw = dsa.dsa_indexer_scores_backward(s["q_idx"], s["q_scale"], s["k_idx"], s["k_scale"], s["w"], s["idx"], s["dsel"])
    return {"dq": dq, "dk": dk, "dw": dw}


# ------------------------------------------------------------------------------------------------- work and exact values
def _entries(case):
    """Selected entries of all rows."""
    rows = [r for r in range(case["T"]) if not case["blank"] or r % case["blank"]]
    return sum(min(case["k"], case["first"] + r + 1) for r in rows)


def work(case):
    T = case["T"]
    if case["op"] == "rope":
        size = 2 if case["dtype"] == "bf16" else 4
        return {"bytes": 2 * T * case["H"] * case["D"] * size + 4 * T + 4 * case["rot"], "flops": 4 * T * case["H"] * case["rot"]}
    S, k, n = case["first"] + T, case["k"], _entries(case)
    read = min(S, n)                                             # rows of the cache that some row selects, at most
    if case["op"] == "index":
        hi, di = case["heads"], case["dim"]
        return {"bytes": T * hi * di * 3 + T * hi * 8 + T * k * 8 + read * (di + 4) + S * di * 2 + 4 * T, "flops": 6 * n * hi * di}
    H = case["H"]
    if case["op"] == "kl":
        return {"bytes": T * H * (D * 2 + 4) + T * k * 12 + read * D * 2 + 4 * T, "flops": 2 * n * H * D}
    return {"bytes": T * H * (4 * D + 4 * D_V + 4) + T * k * 4 + read * D * 2 + S * D * 2, "flops": 2 * n * H * (3 * D + 2 * D_V)}


def exact(case, seed):
    """The definitions in 64 bits, a few rows at a time; the rotation as a product of complex numbers."""
    s = prepare(case, seed)
    T = case["T"]
    if case["op"] == "rope":
        r, off, x = case["rot"], case["off"], s["x"].double()
        turn = torch.polar(torch.full((), s["mscale"], dtype=torch.float64, device="cuda"), s["pos"].double()[:, None] * s["freq"])
        turn = (turn.conj() if case["backward"] else turn)[:, None]
        part = x[..., off:off + r].unflatten(-1, (r // 2, 2) if case["interleaved"] else (2, r // 2))
        if not case["interleaved"]:
            part = part.transpose(-1, -2)
        z = torch.view_as_real(torch.view_as_complex(part.contiguous()) * turn)
        x[..., off:off + r] = (z if case["interleaved"] else z.transpose(-1, -2)).flatten(-2)
        return x
    S, step = case["first"] + T, 64
    parts = []
    into = torch.zeros(S, case["dim"] if case["op"] == "index" else D, dtype=torch.float64, device="cuda")
    for a in range(0, T, step):
        b = slice(a, min(T, a + step))
        ids = s["idx"][b]
        on = (ids >= 0).double()
        at = ids.long() * (ids >= 0)
        if case["op"] == "index":
            q, k = s["q_idx"][b].double(), s["k_idx"].float()[at].double()
            if case["scaled"]:
                q, k = q * s["q_scale"][b].double()[:, None, None], k * s["k_scale"][at].double()[..., None]
            z = torch.einsum("thd,tkd->tkh", q, k)
            up = (s["dsel"][b].double() * on)[..., None] * (z > 0)
            parts.append((torch.einsum("tkh,th,tkd->thd", up, s["w"][b].double(), k), (up * z).sum(1)))
            each = torch.einsum("tkh,thd->tkd", up * s["w"][b].double()[:, None], q)
        else:
            q, rows = s["q"][b].double(), s["c"][at].double()
            x = torch.einsum("thd,tkd->tkh", q, rows) * SCALE
            p = torch.exp(torch.where(on[..., None] > 0, x - s["lse"][b].double()[:, None], -1e9)) * on[..., None]
            if case["op"] == "kl":
                total = p.sum(2) / p.sum((1, 2)).clamp(min=1e-300)[:, None]
                e = torch.softmax(torch.where(on > 0, s["sel"][b].double(), -1e300), 1)
                parts.append(s["dkl"][b].double()[:, None] * (e - total) * on)
                continue
            do = s["dout"][b].double()
            dp = torch.einsum("thd,tkd->tkh", do, rows[..., :D_V])
            ds = SCALE * p * (dp - torch.einsum("thd,thd->th", do, s["out"][b].double())[:, None])
            parts.append(torch.einsum("tkh,tkd->thd", ds, rows))
            each = torch.einsum("tkh,thd->tkd", ds, q)
            each[..., :D_V] += torch.einsum("tkh,thd->tkd", p, do)
        into.index_add_(0, at.flatten(), each.flatten(0, 1))
    if case["op"] == "kl":
        return torch.cat(parts)
    if case["op"] == "attn":
        return {"dq": torch.cat(parts), "dc": into}
    return {"dq": torch.cat([p[0] for p in parts]), "dk": into, "dw": torch.cat([p[1] for p in parts])}
