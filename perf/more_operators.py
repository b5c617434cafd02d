"""The operators of self-attention between a model's NVFP4 linear layers, as measured cases: the
norms and position rotation of queries and keys with their gradient, and softmax attention with its
gradient, which recomputes the probabilities.  The recipe keeps attention in BF16.

`run` computes an operator in its plain form (elementary torch operations in FP32, angles in FP64,
rounded once at the end), or, with `own` set, through the framework.  `exact` computes the same from
the definitions in 64 bits."""
import math

import torch

own = False

BF16, F32 = "bf16", "f32"
TYPES = {BF16: torch.bfloat16, F32: torch.float32}
IDS = {32: torch.int32, 64: torch.int64}
EPS = 1e-6


# ------------------------------------------------------------------------------------------ cases
def rope(T, Hq, Hkv, D, grad, rot=None, interleaved=False, act=BF16, weights=BF16, far=0, base=1e6,
         ids=64, **kw):
    """Positions start at `far` and, of many tokens, again in each of a few documents."""
    return dict(op="rope", T=T, Hq=Hq, Hkv=Hkv, D=D, rot=D if rot is None else rot, grad=grad,
                interleaved=interleaved, act=act, weights=weights, far=far, base=base, ids=ids, **kw)


def attn(T, Hq, Hkv, D, grad, causal=True, window=0, batch=1, keys=0, docs=0, **kw):
    """T queries of each of `batch` sequences over as many keys (or `keys`), or, with docs, T tokens
    of that many documents one after the other."""
    return dict(op="attn", T=T, Hq=Hq, Hkv=Hkv, D=D, grad=grad, causal=causal, window=window,
                batch=batch, keys=keys or T, docs=docs, **kw)


def listed():
    return [
        # one generated token's queries and keys at a far position: latency only
        rope(1, 32, 8, 128, False, far=100000, name="rope_one"),
        # an FP32 model's odd batch, a part of a narrow head rotated in adjacent pairs
        rope(1003, 6, 6, 80, False, rot=36, interleaved=True, act=F32, weights=F32, base=1e4, ids=32,
             name="rope_odd"),
        # the benchmark's tokens and hidden size (40 heads of 128), eight key heads
        rope(8192, 40, 8, 128, False, name="rope_tokens"),
        # a small model's backward pass
        rope(777, 12, 4, 64, True, weights=F32, base=1e4, ids=32, name="rope_grad_small"),
        # the gradient of the benchmark's tokens
        rope(8192, 40, 8, 128, True, name="rope_grad_tokens"),
        # one generated token over the keys so far
        attn(1, 32, 8, 128, False, keys=4097, name="attn_one"),
        # scoring a prompt, nothing to train
        attn(1503, 16, 2, 64, False, name="attn_prompt"),
        # the benchmark's tokens and hidden size, each token over the last 1024
        attn(8192, 40, 8, 128, False, window=1024, name="attn_window"),
        # a small bidirectional model's step: odd lengths, a head of 80
        attn(257, 8, 8, 80, True, causal=False, batch=4, name="attn_train_small"),
        # documents of very different lengths packed into one row of tokens
        attn(4099, 16, 4, 64, True, docs=37, name="attn_train_packed"),
        # the benchmark's tokens and hidden size as one sequence
        attn(8192, 40, 8, 128, True, name="attn_train_large"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    Hkv = rng.choice([1, 2, 3, 4, 8])
    Hq = Hkv * rng.choice([1, 2, 3, 4, 5])
    if rng.random() < 0.4:
        D = 2 * _log(rng, 8, 128)
        if rng.random() < 0.6:
            D = max(16, D // 16 * 16)
        rot = D if rng.random() < 0.6 else 2 * rng.randint(1, D // 2)
        return rope(_log(rng, 1, 8192), Hq, Hkv, D, rng.random() < 0.5, rot=rot,
                    interleaved=rng.random() < 0.5, act=rng.choice([BF16, F32]),
                    weights=rng.choice([BF16, F32]), far=rng.choice([0, 0, 1000, 1000000]),
                    base=rng.choice([1e4, 1e6]), ids=rng.choice([32, 64]))
    D = rng.choice([32, 40, 64, 72, 80, 96, 112, 128, 128])
    T, grad, causal = _log(rng, 1, 8192), rng.random() < 0.6, rng.random() < 0.7
    kind = rng.choice(["one", "batch", "docs", "keys"])
    kw = {}
    if kind == "batch":
        kw["batch"] = rng.randint(2, 8)
        T = max(1, T // kw["batch"])
    elif kind == "docs":
        kw["docs"] = min(T, _log(rng, 2, 64))
    elif kind == "keys":
        kw["keys"] = max(T, _log(rng, 1, 8192))
    if causal and rng.random() < 0.3:
        kw["window"] = _log(rng, 1, 4096)
    most = work(listed()[-1])["flops"]
    while True:
        c = attn(T, Hq, Hkv, D, grad, causal=causal, **kw)
        if c["batch"] * Hq * c["T"] * c["keys"] * D * (14 if grad else 4) <= most:
            return c
        if "keys" in kw:
            kw["keys"] = max(kw["keys"] // 2, T // 2)
        T = max(kw.get("docs", 1), T // 2)


def _lengths(c):
    """Tokens of each document: a few long ones, many short, the same whatever the seed."""
    n, left, out = c["docs"], c["T"], []
    for i in range(n):
        rest = n - 1 - i
        share = ((i * 7919 + 104729) % 1009) / 1009.0
        out.append(left if rest == 0 else
                   min(left - rest, max(1, int(left * share ** 3 * min(1.0, 8.0 / (rest + 1))))))
        left -= out[-1]
    return out


def _pairs(c):
    """Queries and keys that meet, over all sequences."""
    total = 0
    for tq, tk in ([(n, n) for n in _lengths(c)] if c["docs"] else [(c["T"], c["keys"])] * c["batch"]):
        if not c["causal"]:
            total += tq * tk
            continue
        w = c["window"] or tk
        # query i sees keys up to i + tk - tq, the last w of them
        full = max(0, min(tq, tk - w))             # queries with more than w keys behind them
        rest = tq - full                           # these see tk - tq + 1 .. keys
        first = tk - tq + 1
        total += full * w + rest * first + rest * (rest - 1) // 2
    return total


# ----------------------------------------------------------------------------------------- inputs
def _normal(g, *shape, std=1.0, dtype=torch.bfloat16):
    return torch.empty(*shape, dtype=dtype, device="cuda").normal_(0.0, std, generator=g)


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    c = dict(case)
    T, Hq, Hkv, D = c["T"], c["Hq"], c["Hkv"], c["D"]
    if c["op"] == "rope":
        act, wt = TYPES[c["act"]], TYPES[c["weights"]]
        # queries and keys lie in the rows of the projection that makes them, with the values behind
        qkv = _normal(g, T, (Hq + 2 * Hkv) * D, dtype=act)
        q, k = qkv[:, :Hq * D].view(T, Hq, D), qkv[:, Hq * D:(Hq + Hkv) * D].view(T, Hkv, D)
        wq, wk = ((1 + _normal(g, D, std=0.2, dtype=torch.float32)).to(wt) for _ in range(2))
        pos = c["far"] + torch.arange(T, device="cuda") % max(1, (T + 2) // 3)
        inv = (c["base"] ** (-torch.arange(0, c["rot"], 2, dtype=torch.float64) / c["rot"])).float().cuda()
        s = dict(c, q=q, k=k, wq=wq, wk=wk, pos=pos.to(IDS[c["ids"]]), inv=inv)
        if c["grad"]:
            s.update(dq=_normal(g, T, Hq, D, std=1e-2, dtype=act), dk=_normal(g, T, Hkv, D, std=1e-2, dtype=act))
        return s
    if c["keys"] == T:   # queries and keys after their norms, values still in the projection's rows
        shape = (T,) if c["docs"] else (c["batch"], T)
        qkv = _normal(g, *shape, (Hq + 2 * Hkv) * D)
        v = qkv[..., (Hq + Hkv) * D:].view(*shape, Hkv, D)
        q, k = _normal(g, *shape, Hq, D, std=1.2), _normal(g, *shape, Hkv, D, std=1.2)
    else:
        q = _normal(g, c["batch"], T, Hq, D, std=1.2)
        k, v = _normal(g, c["batch"], c["keys"], Hkv, D, std=1.2), _normal(g, c["batch"], c["keys"], Hkv, D)
    cu = None
    if c["docs"]:
        cu = torch.tensor([0] + _lengths(c)).cumsum(0).to(torch.int32).cuda()
    return dict(c, q=q, k=k, v=v, cu=cu, do=_normal(g, *q.shape, std=1e-2) if c["grad"] else None)


# --------------------------------------------------------------------------------------- one pass
def run(s):
    if own:
        return _own(s)
    return _plain_rope(s) if s["op"] == "rope" else _plain_attn(s)


def _own(s):
    import bit_microscaled_numerics_amd as nv
    if s["op"] == "rope":
        rest = (s["q"], s["k"], s["wq"], s["wk"], s["pos"], s["inv"])
        kw = dict(eps=EPS, interleaved=s["interleaved"])
        if not s["grad"]:
            q, k = nv.qk_norm_rope(*rest, **kw)
            return {"q": q, "k": k}
        dq, dk, dwq, dwk = nv.qk_norm_rope_grad(s["dq"], s["dk"], *rest, **kw)
        return {"dq": dq, "dk": dk, "dwq": dwq, "dwk": dwk}
    kw = dict(causal=s["causal"], window=s["window"], cu_q=s["cu"])
    out, lse = nv.attention(s["q"], s["k"], s["v"], **kw)
    if not s["grad"]:
        return {"out": out, "lse": lse}
    dq, dk, dv = nv.attention_grad(s["do"], s["q"], s["k"], s["v"], out, lse, **kw)
    return {"out": out, "lse": lse, "dq": dq, "dk": dk, "dv": dv}


def _split(x, rot, interleaved):
    """The two values of each rotated pair, and the rest of the row."""
    if interleaved:
        return x[..., 0:rot:2], x[..., 1:rot:2], x[..., rot:]
    return x[..., :rot // 2], x[..., rot // 2:rot], x[..., rot:]


def _join(a, b, rest, interleaved):
    pairs = torch.stack((a, b), -1).flatten(-2) if interleaved else torch.cat((a, b), -1)
    return torch.cat((pairs, rest), -1)


def _rotated(x, cos, sin, s):
    a, b, rest = _split(x, s["rot"], s["interleaved"])
    return _join(a * cos - b * sin, b * cos + a * sin, rest, s["interleaved"])


def _plain_rope(s):
    angle = (s["pos"].double().unsqueeze(1) * s["inv"].double()).unsqueeze(1)
    cos, sin = torch.cos(angle).float(), torch.sin(angle).float()
    sides = [("q", s["q"], s["wq"]), ("k", s["k"], s["wk"])]
    res = {}
    for name, x, w in sides:
        n = x.float()
        r = torch.rsqrt((n * n).mean(-1, keepdim=True) + EPS)
        n = n * r
        if not s["grad"]:
            res[name] = _rotated(n * w.float(), cos, sin, s).to(x.dtype)
            continue
        dz = _rotated(s["d" + name].float(), cos, -sin, s)
        res["dw" + name] = (dz * n).sum((0, 1)).to(w.dtype)
        dn = dz * w.float()
        res["d" + name] = (r * (dn - n * (dn * n).mean(-1, keepdim=True))).to(x.dtype)
    return res


def _plain_attn(s):
    """Each sequence by itself, all its heads at once or, of a long one, some."""
    q, k, v, do, D = s["q"], s["k"], s["v"], s["do"], s["D"]
    Hq, Hkv, scale = s["Hq"], s["Hkv"], 1.0 / math.sqrt(D)
    G = Hq // Hkv
    out = torch.empty_like(q)
    lse = torch.empty(q.shape[:-1], dtype=torch.float32, device=q.device)
    dq, dk, dv = (torch.empty(x.shape, dtype=x.dtype, device=x.device) if s["grad"] else None for x in (q, k, v))
    if s["docs"]:
        ends, at = [], 0
        for n in _lengths(s):
            ends.append(slice(at, at + n))
            at += n
    else:
        ends = range(s["batch"])
    for b in ends:
        Tq, Tk = q[b].shape[0], k[b].shape[0]
        hidden = None
        if s["causal"]:
            i = torch.arange(Tk - Tq, Tk, device=q.device).unsqueeze(1)
            j = torch.arange(Tk, device=q.device)
            hidden = j > i
            if s["window"]:
                hidden = hidden | (j <= i - s["window"])
        step = max(1, min(Hkv, (1 << 30) // (G * Tq * Tk)))
        for h in range(0, Hkv, step):
            n = min(step, Hkv - h)
            kv = slice(h, h + n)
            heads = slice(h * G, (h + n) * G)
            q3 = q[b][:, heads].float().reshape(Tq, n, G, D).permute(1, 2, 0, 3).reshape(n, G * Tq, D)
            k3, v3 = (x[b][:, kv].float().transpose(0, 1).contiguous() for x in (k, v))
            z = (q3 @ k3.transpose(1, 2)).mul_(scale).view(n, G, Tq, Tk)
            if hidden is not None:
                z.masked_fill_(hidden, -math.inf)
            top = z.max(-1, keepdim=True).values
            p = torch.exp(z.sub_(top))
            total = p.sum(-1, keepdim=True)
            p.div_(total)
            o = p.view(n, G * Tq, Tk) @ v3
            out[b][:, heads] = o.view(n * G, Tq, D).transpose(0, 1).to(q.dtype)
            lse[b][:, heads] = (top + torch.log(total)).view(n * G, Tq).t()
            if not s["grad"]:
                continue
            g3 = do[b][:, heads].float().reshape(Tq, n, G, D).permute(1, 2, 0, 3).reshape(n, G * Tq, D)
            p = p.view(n, G * Tq, Tk)
            dv[b][:, kv] = (p.transpose(1, 2) @ g3).transpose(0, 1).to(v.dtype)
            ds = (g3 @ v3.transpose(1, 2)).sub_((g3 * o).sum(-1, keepdim=True)).mul_(p)
            dk[b][:, kv] = (ds.transpose(1, 2) @ q3).mul_(scale).transpose(0, 1).to(k.dtype)
            dq3 = (ds @ k3).mul_(scale).view(n * G, Tq, D)
            dq[b][:, heads] = dq3.transpose(0, 1).to(q.dtype)
    res = {"out": out, "lse": lse}
    return dict(res, dq=dq, dk=dk, dv=dv) if s["grad"] else res


# ----------------------------------------------------------------------------- the least of a pass
def work(case):
    c = case
    size = {BF16: 2, F32: 4}
    T, Hq, Hkv, D = c["T"], c["Hq"], c["Hkv"], c["D"]
    if c["op"] == "rope":
        n = T * (Hq + Hkv) * D
        rest = T * (c["ids"] // 8) + 2 * D * size[c["weights"]] * (2 if c["grad"] else 1) + 2 * c["rot"]
        return {"bytes": (3 if c["grad"] else 2) * n * size[c["act"]] + rest, "flops": (14.0 if c["grad"] else 7.0) * n}
    ends = c["batch"] * (T * Hq * 2 + c["keys"] * Hkv * 2) * D * 2
    if c["grad"]:   # q, k, v, do in; out, dq, dk, dv back
        ends = c["batch"] * (T * Hq * 4 + c["keys"] * Hkv * 4) * D * 2
    return {"bytes": ends + c["batch"] * T * Hq * 4, "flops": (14.0 if c["grad"] else 4.0) * _pairs(c) * D * Hq}


# ------------------------------------------------------------------ the definitions, in 64 bits
def exact(case, seed):
    s = prepare(case, seed)
    return _exact_rope(s) if s["op"] == "rope" else _exact_attn(s)


def _exact_rope(s):
    """The rotated pairs as complex numbers times e^(i t), the gradient as autograd finds it."""
    turn = torch.polar(torch.ones((), dtype=torch.float64, device="cuda"),
                       s["pos"].double()[:, None, None] * s["inv"].double())
    res = {}
    for name in ("q", "k"):
        x = s[name].double().requires_grad_(s["grad"])
        w = s["w" + name].double().requires_grad_(s["grad"])
        with torch.set_grad_enabled(s["grad"]):
            z = x * w / torch.sqrt(x.square().sum(-1, keepdim=True) / s["D"] + EPS)
            head = z[..., :s["rot"]]
            pairs = (head.unflatten(-1, (-1, 2)) if s["interleaved"] else
                     head.unflatten(-1, (2, -1)).transpose(-1, -2)).contiguous()
            y = torch.view_as_real(torch.view_as_complex(pairs) * turn)
            y = (y if s["interleaved"] else y.transpose(-1, -2)).flatten(-2)
            y = torch.cat((y, z[..., s["rot"]:]), -1)
        if s["grad"]:
            res["d" + name], res["dw" + name] = torch.autograd.grad(y, (x, w), s["d" + name].double())
        else:
            res[name] = y
    return {n: res[n] for n in (("dq", "dk", "dwq", "dwk") if s["grad"] else ("q", "k"))}


def _exact_attn(s):
    """Head by head; the gradient as autograd finds it."""
    G, grad = s["Hq"] // s["Hkv"], s["grad"]
    names = ("out", "lse", "dq", "dk", "dv") if grad else ("out", "lse")
    like = {"out": s["q"], "lse": s["q"][..., 0], "dq": s["q"], "dk": s["k"], "dv": s["v"]}
    res = {n: torch.zeros(like[n].shape, dtype=torch.float64, device="cuda") for n in names}
    bounds = s["cu"].tolist() if s["docs"] else None
    for b in (slice(*e) for e in zip(bounds, bounds[1:])) if s["docs"] else range(s["batch"]):
        Tq, Tk = s["q"][b].shape[0], s["k"][b].shape[0]
        seen = None
        if s["causal"]:
            seen = torch.ones(Tq, Tk, dtype=torch.bool, device="cuda").tril(Tk - Tq)
            if s["window"]:
                seen = seen.triu(Tk - Tq - s["window"] + 1)
        for h in range(s["Hq"]):
            args = [x[b][:, i].double().requires_grad_(grad) for x, i in
                    ((s["q"], h), (s["k"], h // G), (s["v"], h // G))]
            with torch.set_grad_enabled(grad):
                z = (args[0] / math.sqrt(s["D"])) @ args[1].T
                if seen is not None:
                    z = z.where(seen, -math.inf)
                lse = torch.logsumexp(z, 1)
                o = torch.exp(z - lse[:, None]) @ args[2]
            res["out"][b][:, h] = o.detach()
            res["lse"][b][:, h] = lse.detach()
            if grad:
                dq, dk, dv = torch.autograd.grad(o, args, s["do"][b][:, h].double())
                res["dq"][b][:, h] = dq
                res["dk"][b][:, h // G] += dk
                res["dv"][b][:, h // G] += dv
            del z, o
    return res
