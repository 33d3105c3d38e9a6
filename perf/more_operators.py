"""Measured cases of linear attention with a decay for each head (forward, training pass,
decode step) and of the group norm with an activation behind it (forward, training pass).

``run`` computes one pass in plain torch operations, or, where ``own`` is true, by the calls
a user of the package makes."""
import math

import torch

own = False

EPS = 1e-5               # the norm's epsilon
CHUNK = 128              # tokens of a chunk of the plain form


# ------------------------------------------------------------------------------- the cases

def listed():
    return [
        # latency of one short prompt, a fixed decay for each head
        dict(name="lin small f32", op="lin", io="f32", batch=1, L=64, H=4, Hk=4, K=64, V=64, decay="fixed"),
        # prefill of one long prompt
        dict(name="lin prompt bf16", op="lin", io="bf16", batch=1, L=16384, H=32, Hk=32, K=128, V=128, decay="fixed"),
        # queries and keys shared by all heads, a decay per token: the widths of the 2.7B scalar-decay layer
        dict(name="lin shared bf16", op="lin", io="bf16", batch=4, L=8192, H=80, Hk=1, K=128, V=64, decay="token"),
        # sizes that fill no tile
        dict(name="lin odd f32", op="lin", io="f32", batch=3, L=777, H=5, Hk=5, K=80, V=100, decay="token"),
        # a training step's layer on packed documents
        dict(name="train packed bf16", op="train", io="bf16", batch=4, L=4096, H=16, Hk=16, K=128, V=128, decay="packed"),
        # the same in fp32 with shared heads, at sizes that fill no tile
        dict(name="train odd f32", op="train", io="f32", batch=2, L=333, H=6, Hk=2, K=40, V=72, decay="fixed"),
        # decode: a batch on slots at the 2.7B widths, beams and padding among it; one sequence at 130M widths
        dict(name="step 64 bf16", op="step", io="bf16", batch=64, H=80, Hk=1, K=128, V=64, slots=True),
        dict(name="step one f32", op="step", io="f32", batch=1, H=24, Hk=24, K=128, V=64, slots=False),
        # the layer's output stage: each head's output normalised, times the gate; a long prompt and one token
        dict(name="norm long bf16", op="norm", io="bf16", rows=16384, groups=32, width=128, gate=True, act="silu", affine=True),
        dict(name="norm one f32", op="norm", io="f32", rows=1, groups=24, width=64, gate=True, act="silu", affine=True),
        # its training pass at the width of the long-context scan, and where neither rows nor groups fill anything
        dict(name="norm train bf16", op="ntrain", io="bf16", rows=16384, groups=40, width=64, gate=True, act="silu", affine=True),
        dict(name="norm train odd f32", op="ntrain", io="f32", rows=1537, groups=3, width=257, gate=False, act="silu", affine=True),
    ]


def _spread(rng, lo, hi):
    """A whole number between lo and hi, spread over its logarithm."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["lin", "lin", "lin", "train", "train", "train", "step", "step", "norm", "ntrain"])
    io = rng.choice(["f32", "bf16"])
    if op in ("lin", "train"):
        most, long = (24 << 20, 16384) if op == "lin" else (8 << 20, 4096)
        while True:
            Hk, share = _spread(rng, 1, 32), rng.choice([1, 1, 2, 4])
            c = dict(op=op, io=io, batch=_spread(rng, 1, 8), L=_spread(rng, 1, long), H=Hk * share, Hk=Hk,
                     K=rng.choice([64, 128, _spread(rng, 4, 256)]), V=rng.choice([64, 128, _spread(rng, 4, 256)]),
                     decay=rng.choice(["fixed", "token", "packed"]))
            if c["batch"] * c["L"] * c["H"] * (c["K"] + c["V"]) <= most:
                return c
    if op == "step":
        while True:
            Hk, share = _spread(rng, 1, 32), rng.choice([1, 1, 2, 4])
            c = dict(op=op, io=io, batch=_spread(rng, 1, 256), H=Hk * share, Hk=Hk, K=rng.choice([64, 128, _spread(rng, 4, 256)]),
                     V=rng.choice([64, 128, _spread(rng, 4, 256)]), slots=rng.random() < 0.6)
            if c["batch"] * c["H"] * c["K"] * c["V"] <= 32 << 20:
                return c
    while True:
        c = dict(op=op, io=io, rows=_spread(rng, 1, 20000), groups=_spread(rng, 1, 64), width=rng.choice([64, 128, _spread(rng, 4, 4096)]),
                 gate=rng.random() < 0.6, act=rng.choice(["silu", "silu", "none"]), affine=rng.random() < 0.8)
        if c["rows"] * c["groups"] * c["width"] <= 24 << 20:
            return c


def work(case):
    c = case
    es = 2 if c["io"] == "bf16" else 4
    if c["op"] in ("lin", "train"):
        n, state = c["batch"] * c["L"], 4 * c["batch"] * c["H"] * c["K"] * c["V"]
        qk, v = n * c["Hk"] * c["K"] * es, n * c["H"] * c["V"] * es
        g = 4 * (c["H"] if c["decay"] == "fixed" else n * c["H"])
        # a product with the state and its update, and the pairs of a chunk of 64 tokens
        flops = n * c["H"] * (4 * c["K"] * c["V"] + 64 * (c["K"] + c["V"]))
        if c["op"] == "lin":          # q, k, v in, o out; the states at both ends
            return {"bytes": 2 * qk + 2 * v + g + 2 * state, "flops": flops}
        # forward as above; backward: q, k, v, do in, dq, dk, dv out; two more states
        return {"bytes": 2 * qk + 2 * v + 2 * state + 4 * qk + 3 * v + 3 * g + 3 * state, "flops": int(3.5 * flops)}
    if c["op"] == "step":
        n = c["batch"] * c["H"]
        return {"bytes": n * (8 * c["K"] * c["V"] + 2 * c["V"] * es) + 2 * c["batch"] * c["Hk"] * c["K"] * es,
                "flops": n * 5 * c["K"] * c["V"]}
    n = c["rows"] * c["groups"] * c["width"]
    if c["op"] == "norm":
        return {"bytes": n * es * (3 if c["gate"] else 2), "flops": 12 * n}
    return {"bytes": n * es * (8 if c["gate"] else 5), "flops": 40 * n}


# ------------------------------------------------------------------------------ the inputs

def prepare(case, seed):
    c = dict(case)
    gen = torch.Generator(device="cuda").manual_seed(int(seed) * 1000003 + 29)
    io = torch.bfloat16 if c["io"] == "bf16" else torch.float32
    n = lambda *shape: torch.randn(shape, generator=gen, device="cuda")             # noqa: E731
    u = lambda *shape: torch.rand(shape, generator=gen, device="cuda")              # noqa: E731
    s = dict(c)
    if c["op"] in ("norm", "ntrain"):
        rows, C = c["rows"], c["groups"] * c["width"]
        # outputs of heads: each of its own size, off its zero
        head = torch.exp(n(c["groups"], 1)).expand(c["groups"], c["width"]).reshape(C)
        s["x"] = ((n(rows, C) + 0.5 * n(C)) * head).to(io)
        s["z"] = n(rows, C).to(io) if c["gate"] else None
        s["weight"] = 1 + 0.1 * n(C) if c["affine"] else None
        s["bias"] = 0.1 * n(C) if c["affine"] else None
        if c["op"] == "ntrain":
            s["dy"] = n(rows, C).to(io)
        return s
    B, H, Hk, K, V = c["batch"], c["H"], c["Hk"], c["K"], c["V"]
    s["scale"] = K ** -0.5
    # half lives of heads from 20 tokens to some hundreds
    fixed = torch.log1p(-torch.exp2(-5 - 4 * torch.arange(H, device="cuda") / max(1, H - 1)))
    if c["op"] == "step":
        s["q"], s["k"], s["v"] = n(B, Hk, K).to(io), n(B, Hk, K).to(io), n(B, H, V).to(io)
        s["g"] = fixed * (0.5 + u(B, H))
        s["state"] = 3 * n(2 * B if c["slots"] else B, H, K, V)
        s["o"] = torch.zeros(B, H, V, dtype=io, device="cuda")
        s["read"] = s["write"] = None
        s["live"] = torch.arange(B, device="cuda")
        if c["slots"]:
            # beams read their parents' slots (a parent may be shared, -1: a sequence that starts)
            # and write slots of their own; the last rows of a padded batch have none
            perm = torch.randperm(2 * B, generator=gen, device="cuda").to(torch.int32)
            parents, write = perm[:B].clone(), perm[B:].clone()
            if B > 2:
                parents[1] = parents[0]
                parents[2] = -1
            pad = B // 8
            if pad:
                write[B - pad:] = -1
            s["read"], s["write"], s["live"] = parents, write, s["live"][: B - pad]
        return s
    L = c["L"]
    s["q"], s["k"], s["v"] = n(B, L, Hk, K).to(io), n(B, L, Hk, K).to(io), n(B, L, H, V).to(io)
    s["g"] = fixed if c["decay"] == "fixed" else fixed * torch.exp(n(B, L, H))
    if c["decay"] == "packed":                                # documents start anew
        s["g"] = s["g"].masked_fill((u(B, L) < 4.0 / max(L, 8))[..., None], -math.inf)
    s["h0"] = n(B, H, K, V)
    if c["op"] == "train":
        s["do"], s["dlast"] = n(B, L, H, V).to(io), n(B, H, K, V)
    return s


# -------------------------------------------------------------------------- the plain forms

def _chunks(t, share, nc):
    """[batch, L, heads, width] as fp32 [batch, H, chunks, CHUNK, width], padded with zeros."""
    t = t.float()
    t = torch.nn.functional.pad(t, (0, 0, 0, 0, 0, nc * CHUNK - t.shape[1]))
    t = t.repeat_interleave(share, 2) if share > 1 else t
    return t.unflatten(1, (nc, CHUNK)).permute(0, 3, 1, 2, 4).contiguous()


def _decays(d, same):
    return torch.exp(torch.where(same, d, -math.inf)).float()


def _plain_lin(s, train):
    io, share = s["q"].dtype, s["H"] // s["Hk"]
    L, H = s["L"], s["H"]
    nc = -(-L // CHUNK)
    q, k, v = _chunks(s["q"], share, nc) * s["scale"], _chunks(s["k"], share, nc), _chunks(s["v"], 1, nc)
    # logarithms of the decays since the start, in 64 bits (their differences count), and how often
    # the state has started anew
    g = s["g"].double().expand(s["batch"], L, H).transpose(1, 2)
    g = torch.nn.functional.pad(g, (0, nc * CHUNK - L))
    anew = torch.isinf(g)
    run = anew.long().cumsum(-1).unflatten(-1, (nc, CHUNK))
    c = g.masked_fill(anew, 0.0).cumsum(-1).unflatten(-1, (nc, CHUNK))
    end, rend = c[..., -1], run[..., -1]
    first, rfirst = torch.nn.functional.pad(end, (1, 0))[..., :-1], torch.nn.functional.pad(rend, (1, 0))[..., :-1]
    tril = torch.ones(CHUNK, CHUNK, dtype=torch.bool, device=q.device).tril()
    D = _decays(c[..., :, None] - c[..., None, :], tril & (run[..., :, None] == run[..., None, :]))
    f = _decays(c - first[..., None], run == rfirst[..., None])[..., None]       # since the chunk's start
    w = _decays(end[..., None] - c, run == rend[..., None])[..., None]           # to its end
    # from the end of chunk m to the start of chunk n, from the start of all to it, and to the end of all
    before = torch.ones(nc, nc, dtype=torch.bool, device=q.device).tril(-1)
    M = _decays(first[..., :, None] - end[..., None, :], before & (rfirst[..., :, None] == rend[..., None, :]))
    M0 = _decays(first, rfirst == 0)[..., None, None]
    ML = _decays(end[..., -1:] - end, rend == rend[..., -1:])[..., None, None]
    own_end = torch.matmul((w * k).transpose(-1, -2).contiguous(), v)            # each chunk's own state
    start = torch.matmul(M, own_end.flatten(-2)).unflatten(-1, own_end.shape[-2:]) + M0 * s["h0"][:, :, None]
    through = _decays(end - first, rend == rfirst)[..., None, None]
    ends = through * start + own_end
    P = torch.matmul(q, k.transpose(-1, -2).contiguous()) * D
    o = torch.matmul(P, v) + f * torch.matmul(q, start)
    back = lambda t: t.permute(0, 2, 3, 1, 4).flatten(1, 2)[:, :L]                # noqa: E731
    out = {"o": back(o).to(io), "last": ends[:, :, -1].clone()}
    if not train:
        return out
    do = _chunks(s["do"], 1, nc)
    own_first = torch.matmul((f * q).transpose(-1, -2).contiguous(), do)         # at each chunk's start
    R = torch.matmul(M.transpose(-1, -2).contiguous(), own_first.flatten(-2)).unflatten(-1, own_first.shape[-2:])
    R = R + ML * s["dlast"][:, :, None]                                          # gradient of the state at a chunk's end
    dP = torch.matmul(do, v.transpose(-1, -2).contiguous()) * D
    dq = torch.matmul(dP, k) + f * torch.matmul(do, start.transpose(-1, -2).contiguous())
    dk = torch.matmul(dP.transpose(-1, -2).contiguous(), q) + w * torch.matmul(v, R.transpose(-1, -2).contiguous())
    dv = torch.matmul(P.transpose(-1, -2).contiguous(), do) + w * torch.matmul(k, R)
    # what passes a token's decay: pairs of the chunk that lie on both sides of it, and what leaves the chunk
    d = ((q.double() * dq).sum(-1) - (k.double() * dk).sum(-1))
    d = d.flip(-1).cumsum(-1).flip(-1) + (ends.double() * R).sum((-1, -2))[..., None]
    d = d.flatten(2).masked_fill(anew, 0.0)[..., :L].transpose(1, 2)
    out["dg"] = (d.sum((0, 1)) if s["g"].dim() == 1 else d).float()
    heads = lambda t: back(t).unflatten(2, (s["Hk"], share)).sum(3)               # noqa: E731
    out["dq"], out["dk"], out["dv"] = (heads(dq) * s["scale"]).to(io), heads(dk).to(io), back(dv).to(io)
    out["dh0"] = own_first[:, :, 0] + through[:, :, 0] * R[:, :, 0]
    return out


def _plain_step(s):
    share = s["H"] // s["Hk"]
    q, k = (s[n].float().repeat_interleave(share, 1) for n in ("q", "k"))
    if s["read"] is None:
        h = s["state"]
    else:
        h = torch.where((s["read"] >= 0)[:, None, None, None], s["state"][s["read"].long().clamp(min=0)], 0.0)
    h = torch.exp(s["g"])[..., None, None] * h + k[..., None] * s["v"].float()[:, :, None]
    o = (s["scale"] * (q[..., None] * h).sum(-2)).to(s["o"].dtype)
    at = s["live"]
    s["state"][at if s["write"] is None else s["write"][at].long()] = h[at]
    s["o"][at] = o[at]
    return {"o": s["o"], "state": s["state"]}


def _plain_norm(s, train):
    io, shape = s["x"].dtype, s["x"].shape
    grouped = lambda t: t.unflatten(1, (s["groups"], s["width"]))                 # noqa: E731
    x = grouped(s["x"].float())
    x = x - x.mean(-1, keepdim=True)
    rstd = torch.rsqrt((x * x).mean(-1, keepdim=True) + EPS)
    xh = (x * rstd).reshape(shape)
    n = xh * s["weight"] + s["bias"] if s["affine"] else xh
    t = n if s["z"] is None else s["z"].float()
    sg = torch.sigmoid(t) if s["act"] == "silu" else torch.ones_like(t)
    act = t * sg
    out = {"y": (act if s["z"] is None else n * act).to(io)}
    if not train:
        return out
    dy = s["dy"].float()
    slope = sg * (1 + t * (1 - sg)) if s["act"] == "silu" else sg
    dn = dy * (slope if s["z"] is None else act)
    if s["z"] is not None:
        out["dz"] = (dy * n * slope).to(io)
    if s["affine"]:
        out["dweight"] = (dn * xh).sum(0, dtype=torch.float64).float()
        out["dbias"] = dn.sum(0, dtype=torch.float64).float()
        dn = dn * s["weight"]
    d, xg = grouped(dn), grouped(xh)
    d = rstd * (d - d.mean(-1, keepdim=True) - xg * (d * xg).mean(-1, keepdim=True))
    out["dx"] = d.reshape(shape).to(io)
    return out


# -------------------------------------------------------------------------------- one pass

def run(state):
    s = state
    if own:
        return _run_own(s)
    if s["op"] in ("lin", "train"):
        return _plain_lin(s, s["op"] == "train")
    return _plain_step(s) if s["op"] == "step" else _plain_norm(s, s["op"] == "ntrain")


def _run_own(s):
    import selective_state_space_s6_amd as ss
    if s["op"] == "step":
        o = ss.linear_attention_step(s["q"], s["k"], s["v"], s["g"], state=s["state"], o=s["o"], scale=s["scale"],
                                     read_slots=s["read"], write_slots=s["write"])
        return {"o": o, "state": s["state"]}
    if s["op"] in ("norm", "ntrain"):
        kind = dict(groups=s["groups"], eps=EPS, activation=s["act"])
        out = {"y": ss.group_norm_fwd(s["x"], s["weight"], s["bias"], s["z"], **kind)}
        if s["op"] == "ntrain":
            d = ss.group_norm_bwd(s["x"], s["weight"], s["bias"], s["z"], dy=s["dy"], **kind)
            out.update((name, d[name]) for name in ("dz", "dweight", "dbias", "dx") if name in d)
        return out
    o, last = ss.linear_attention_fwd(s["q"], s["k"], s["v"], s["g"], scale=s["scale"], initial_state=s["h0"],
                                      return_last_state=True)
    out = {"o": o, "last": last}
    if s["op"] == "train":
        d = ss.linear_attention_bwd(s["q"], s["k"], s["v"], s["g"], do=s["do"], scale=s["scale"], initial_state=s["h0"],
                                    dlast_state=s["dlast"])
        out.update(dg=d["dlog_decay"], dq=d["dq"], dk=d["dk"], dv=d["dv"], dh0=d["dinitial_state"])
    return out


# --------------------------------------------- the definitions in 64 bits, token by token

def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] in ("norm", "ntrain"):
        return _exact_norm(s, case["op"] == "ntrain")
    if case["op"] == "step":
        return _exact_step(s)
    return _exact_lin(s, case["op"] == "train")


def _outer(a, b):
    return a.unsqueeze(-1) * b.unsqueeze(-2)


def _exact_lin(s, train):
    B, L, H, Hk = s["batch"], s["L"], s["H"], s["Hk"]
    head = torch.arange(H, device="cuda") // (H // Hk)
    key = lambda t: s["k"][:, t].double()[:, head]                                # noqa: E731
    query = lambda t: s["q"][:, t].double()[:, head] * s["scale"]                 # noqa: E731
    value = lambda t: s["v"][:, t].double()                                       # noqa: E731

    def decayed(h, t):
        """The state h as it reaches token t."""
        a = torch.exp((s["g"] if s["g"].dim() == 1 else s["g"][:, t]).double())
        return a[..., None, None] * h

    h, o, marks = s["h0"].double(), torch.empty(B, L, H, s["V"], dtype=torch.float64, device="cuda"), []
    for t in range(L):
        if train and t % 64 == 0:
            marks.append(h)
        h = decayed(h, t) + _outer(key(t), value(t))
        o[:, t] = (query(t).unsqueeze(-1) * h).sum(-2)
    out = {"o": o, "last": h}
    if not train:
        return out
    dq, dk = (torch.zeros(B, L, Hk, s["K"], dtype=torch.float64, device="cuda") for _ in range(2))
    dv, dg = torch.empty_like(o), torch.empty(B, L, H, dtype=torch.float64, device="cuda")
    R = s["dlast"].double()
    for first in range((L - 1) // 64 * 64, -1, -64):
        states = [marks[first // 64]]
        for t in range(first, min(L, first + 64)):
            states.append(decayed(states[-1], t) + _outer(key(t), value(t)))
        for t in range(min(L, first + 64) - 1, first - 1, -1):
            dout = s["do"][:, t].double()
            R = R + _outer(query(t), dout)
            dq[:, t].index_add_(1, head, s["scale"] * (states[t - first + 1] * dout.unsqueeze(-2)).sum(-1))
            dk[:, t].index_add_(1, head, (R * value(t).unsqueeze(-2)).sum(-1))
            dv[:, t] = (R * key(t).unsqueeze(-1)).sum(-2)
            dg[:, t] = (R * decayed(states[t - first], t)).sum((-1, -2))
            R = decayed(R, t)
    out["dg"] = dg.sum((0, 1)) if s["g"].dim() == 1 else dg
    out.update(dq=dq, dk=dk, dv=dv, dh0=R)
    return out


def _exact_step(s):
    state, o = s["state"].double(), s["o"].double()
    new, share = state.clone(), s["H"] // s["Hk"]
    for b in range(s["batch"]):
        src = b if s["read"] is None else int(s["read"][b])
        dst = b if s["write"] is None else int(s["write"][b])
        if dst < 0:
            continue
        k, q = (torch.repeat_interleave(s[n][b].double(), share, 0) for n in ("k", "q"))
        h = _outer(k, s["v"][b].double())
        if src >= 0:
            h = h + torch.exp(s["g"][b].double())[:, None, None] * state[src]
        new[dst] = h
        o[b] = torch.matmul(q.unsqueeze(-2), h).squeeze(-2) * s["scale"]
    return {"o": o, "state": new}


def _exact_norm(s, train):
    rows, C = s["x"].shape
    x = s["x"].double().reshape(rows, s["groups"], -1)
    var, mean = torch.var_mean(x, dim=-1, correction=0, keepdim=True)
    xh = ((x - mean) / torch.sqrt(var + EPS)).reshape(rows, C)
    w = s["weight"].double() if s["affine"] else torch.ones(C, dtype=torch.float64, device="cuda")
    b = s["bias"].double() if s["affine"] else 0.0
    n = w * xh + b
    e = (n if s["z"] is None else s["z"].double())
    gate, slope = e, torch.ones_like(e)
    if s["act"] == "silu":
        p = 1 / (1 + torch.exp(-e))
        gate, slope = e * p, p + e * p * (1 - p)
    out = {"y": gate if s["z"] is None else n * gate}
    if not train:
        return out
    dy = s["dy"].double()
    if s["z"] is None:
        dn = dy * slope
    else:
        dn = dy * gate
        out["dz"] = dy * n * slope
    if s["affine"]:
        out["dweight"], out["dbias"] = (dn * xh).sum(0), dn.sum(0)
    dxh, xh = (dn * w).reshape(x.shape), xh.reshape(x.shape)
    inner = s["width"] * dxh - dxh.sum(-1, keepdim=True) - xh * (dxh * xh).sum(-1, keepdim=True)
    out["dx"] = (inner / (s["width"] * torch.sqrt(var + EPS))).reshape(rows, C)
    return out
