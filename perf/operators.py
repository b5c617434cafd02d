"""The operators at the two ends of a language model's training step, and over its gradients, as
measured cases: the token embedding and its gradient, the output head's softmax cross entropy with
its gradient, and the global gradient norm with clipping.  The recipe keeps the embedding, the head
and the gradients in BF16 beside the NVFP4 linear layers.

`run` computes an operator in its plain form (elementary torch operations in FP32, rounded once at
the end), or, with `own` set, through the framework.  `exact` computes the same from the definitions
in 64 bits."""
import math

import torch

own = False

BF16, F32 = "bf16", "f32"
TYPES = {BF16: torch.bfloat16, F32: torch.float32}
IDS = {32: torch.int32, 64: torch.int64}


# ------------------------------------------------------------------------------------------ cases
def ce(T, V, D, grad, ignored=0.0, weighted=False, ids=64, **kw):
    return dict(op="ce", T=T, V=V, D=D, grad=grad, ignored=ignored, weighted=weighted, ids=ids, **kw)


def embed(T, V, D, grad, table=BF16, act=BF16, zipf=True, ids=64, **kw):
    return dict(op="embed", T=T, V=V, D=D, grad=grad, table=table, act=act, zipf=zipf, ids=ids, **kw)


def clip(layers, hidden, ffn, dtype=BF16, out=BF16, flat=False, std=1e-3, **kw):
    return dict(op="clip", layers=layers, hidden=hidden, ffn=ffn, dtype=dtype, out=out, flat=flat,
                std=std, **kw)


def listed():
    return [
        # the log probability of one generated token: the vocabulary matrix is read once, latency counts
        ce(1, 32000, 1024, False, name="ce_score_one"),
        # scoring a short prompt for evaluation, an odd vocabulary, nothing to train
        ce(333, 50257, 2048, False, ids=32, name="ce_score_prompt"),
        # a small model's step: odd tokens and vocabulary, a tenth of the tokens padding
        ce(1003, 32003, 512, True, ignored=0.1, name="ce_train_small"),
        # a fine-tuning batch: most tokens belong to the prompt and carry no loss, the others a weight
        ce(2500, 65536, 2048, True, ignored=0.6, weighted=True, name="ce_train_masked"),
        # the head of the benchmark's model: its tokens and hidden size, a vocabulary of 2^17
        ce(8192, 131072, 5120, True, name="ce_train_large"),
        # one generated token's embedding: one row, latency only
        embed(1, 131072, 5120, False, name="embed_one"),
        # the benchmark's tokens through the benchmark's hidden size
        embed(8192, 131072, 5120, False, name="embed_tokens"),
        # that lookup's gradient, words as frequent as in text: every row of the table is written
        embed(8192, 131072, 5120, True, name="embed_grad_tokens"),
        # many tokens, a small odd vocabulary, FP32 table of an odd width: long runs of one word
        embed(30001, 5003, 771, True, table=F32, ids=32, name="embed_grad_odd"),
        # a small model's gradients as odd pieces of one flat FP32 buffer
        clip(5, 96, 257, dtype=F32, out=F32, flat=True, std=1e-2, name="clip_small"),
        # FP32 gradients from the weight-gradient GEMMs, clipped into BF16
        clip(3, 2048, 8192, dtype=F32, out=BF16, name="clip_to_bf16"),
        # three of the benchmark's FFN blocks, BF16 (2^29 elements and more)
        clip(3, 5120, 20480, name="clip_large"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["ce", "embed", "clip"])
    if op == "ce":
        return ce(_log(rng, 1, 8192), _log(rng, 1000, 131072), 16 * _log(rng, 4, 320),
                  rng.random() < 0.6, ignored=rng.choice([0.0, 0.1, 0.6]),
                  weighted=rng.random() < 0.5, ids=rng.choice([32, 64]))
    if op == "embed":
        V, D = _log(rng, 1000, 131072), _log(rng, 33, 5120)
        if rng.random() < 0.5:
            D = max(16, D // 16 * 16)
        return embed(_log(rng, 1, 32768), V, D, rng.random() < 0.6, table=rng.choice([BF16, F32]),
                     act=rng.choice([BF16, F32]), zipf=rng.random() < 0.7, ids=rng.choice([32, 64]))
    hidden = _log(rng, 17, 5120)
    return clip(rng.randint(1, 3), hidden, _log(rng, hidden, 4 * hidden), dtype=rng.choice([BF16, F32]),
                out=rng.choice([BF16, F32]), flat=rng.random() < 0.5, std=rng.choice([1e-4, 1e-3]))


# ----------------------------------------------------------------------------------------- inputs
def _normal(g, *shape, std=1.0, dtype=torch.bfloat16):
    return torch.empty(*shape, dtype=dtype, device="cuda").normal_(0.0, std, generator=g)


def _ids(g, T, V, zipf, dtype):
    """Word numbers, uniform or with the frequencies 1 / rank of words in text, the ranks spread
    over the vocabulary."""
    u = torch.rand(T, generator=g, device="cuda", dtype=torch.float64)
    if not zipf:
        return (u * V).long().clamp_(max=V - 1).to(dtype)
    rank = torch.exp(u * math.log(V)).long().clamp_(1, V) - 1
    return ((rank * 7919 + 13) % V).to(dtype)


def _clip_shapes(c):
    H, F = c["hidden"], c["ffn"]
    return [s for _ in range(c["layers"]) for s in ((F, H), (H, F), (H,), (H,))] + [(H + 1, 3)]


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    c = dict(case)
    if c["op"] == "ce":
        T, V, D = c["T"], c["V"], c["D"]
        w = _normal(g, V, D, std=0.02)
        t = _ids(g, T, V, True, torch.int64)
        # hidden states that favour their target by 0 .. 12 in the logit, as a trained model's do
        boost = 12.0 * torch.rand(T, 1, generator=g, device="cuda") / (0.0004 * D)
        h = (_normal(g, T, D, dtype=torch.float32) + boost * w[t].float()).to(torch.bfloat16)
        drop = torch.rand(T, generator=g, device="cuda") < c["ignored"]
        t = torch.where(drop, torch.full_like(t, -100), t).to(IDS[c["ids"]])
        weight = torch.rand(T, generator=g, device="cuda") / T if c["weighted"] else None
        return dict(c, h=h, w=w, t=t, weight=weight)
    if c["op"] == "embed":
        T, V, D = c["T"], c["V"], c["D"]
        ids = _ids(g, T, V, c["zipf"], IDS[c["ids"]])
        scale = math.sqrt(D)
        if c["grad"]:
            return dict(c, ids=ids, scale=scale, dy=_normal(g, T, D, std=1e-3, dtype=TYPES[c["act"]]))
        return dict(c, ids=ids, scale=scale, w=_normal(g, V, D, std=0.02, dtype=TYPES[c["table"]]))
    shapes = _clip_shapes(c)
    dt, od = TYPES[c["dtype"]], TYPES[c["out"]]
    if c["flat"]:
        sizes = [math.prod(s) for s in shapes]
        flat = _normal(g, sum(sizes), std=c["std"], dtype=dt)
        grads = [x.view(s) for x, s in zip(flat.split(sizes), shapes)]
    else:
        grads = [_normal(g, *s, std=c["std"], dtype=dt) for s in shapes]
    return dict(c, grads=grads, clipped=[torch.empty(s, dtype=od, device="cuda") for s in shapes])


# --------------------------------------------------------------------------------------- one pass
def run(s):
    if own:
        return _own(s)
    if s["op"] == "ce":
        return _plain_ce(s["h"], s["w"], s["t"].long(), s["weight"], s["grad"])
    if s["op"] == "embed":
        if s["grad"]:
            return _plain_embed_grad(s["ids"].long(), s["dy"], s["V"], s["scale"], TYPES[s["table"]])
        return (s["w"][s["ids"].long()].float() * s["scale"]).to(TYPES[s["act"]])
    return _plain_clip(s["grads"], 1.0, TYPES[s["out"]])


def _own(s):
    import bit_microscaled_numerics_amd as nv
    if s["op"] == "ce":
        if s["grad"]:
            loss, _, dh, dw = nv.linear_ce_grad(s["h"], s["w"], s["t"], row_weight=s["weight"])
            return {"loss": loss, "dh": dh, "dw": dw}
        loss, lse = nv.linear_ce(s["h"], s["w"], s["t"])
        return {"loss": loss, "lse": lse}
    if s["op"] == "embed":
        if s["grad"]:
            return nv.embed_grad(s["ids"], s["dy"], s["V"], s["scale"], dtype=TYPES[s["table"]])
        return nv.embed(s["ids"], s["w"], s["scale"], dtype=TYPES[s["act"]])
    norm = nv.clip_grads(s["grads"], 1.0, out=s["clipped"])
    return {"norm": norm, "grads": s["clipped"]}


def _plain_ce(h, w, t, weight, grad):
    h32, w32 = h.float(), w.float()
    valid = (t >= 0) & (t < w.shape[0])
    at = torch.where(valid, t, torch.zeros_like(t)).unsqueeze(1)
    logits = h32 @ w32.t()
    top = logits.max(dim=1, keepdim=True).values
    target = logits.gather(1, at)
    z = torch.exp(logits.sub_(top))
    total = z.sum(dim=1, keepdim=True)
    lse = torch.log(total) + top
    loss = torch.where(valid, (lse - target).squeeze(1), torch.zeros_like(lse.squeeze(1)))
    if not grad:
        return {"loss": loss, "lse": lse.squeeze(1)}
    if weight is None:
        weight = torch.ones_like(loss) / valid.sum().clamp(min=1)
    p = z.div_(total)
    # p - 1 at the target, as 1 minus a sum of the others would lose nothing: exp(x) - 1 of x = -loss
    p.scatter_(1, at, torch.expm1(target - lse))
    p.mul_(torch.where(valid, weight, torch.zeros_like(weight)).unsqueeze(1))
    return {"loss": loss, "dh": (p @ w32).to(h.dtype), "dw": (p.t() @ h32).to(w.dtype)}


def _plain_embed_grad(ids, dy, V, scale, dtype):
    dw = torch.zeros(V, dy.shape[1], dtype=torch.float32, device=dy.device)
    return dw.index_add_(0, ids, dy.float()).mul_(scale).to(dtype)


def _plain_clip(grads, max_norm, out_dtype):
    norm = torch.sqrt(sum(g.float().square().sum(dtype=torch.float64) for g in grads))
    coef = (max_norm / (norm + 1e-6)).clamp(max=1.0).float()
    return {"norm": norm.float().reshape(1), "grads": [(g.float() * coef).to(out_dtype) for g in grads]}


# ----------------------------------------------------------------------------- the least of a pass
def work(case):
    c = case
    size = {BF16: 2, F32: 4}
    if c["op"] == "ce":
        T, V, D = c["T"], c["V"], c["D"]
        ends = (T + V) * D * 2
        if c["grad"]:
            return {"bytes": 2 * ends + T * (c["ids"] // 8 + 4), "flops": 6.0 * T * V * D}
        return {"bytes": ends + T * (c["ids"] // 8 + 8), "flops": 2.0 * T * V * D}
    if c["op"] == "embed":
        T, V, D = c["T"], c["V"], c["D"]
        rows = V if c["grad"] else T
        return {"bytes": T * D * size[c["act"]] + rows * D * size[c["table"]] + T * (c["ids"] // 8),
                "flops": 1.0 * T * D}
    n = sum(math.prod(s) for s in _clip_shapes(c))
    return {"bytes": n * (size[c["dtype"]] + size[c["out"]]), "flops": 3.0 * n}


# ------------------------------------------------------------------ the definitions, in 64 bits
def exact(case, seed):
    s = prepare(case, seed)
    if s["op"] == "ce":
        return _exact_ce(s)
    if s["op"] == "embed":
        ids = s["ids"].long()
        if not s["grad"]:
            return torch.index_select(s["w"], 0, ids).double() * s["scale"]
        order = torch.argsort(ids)
        run_ends = torch.cumsum(torch.bincount(ids, minlength=s["V"]), 0)
        sums = torch.zeros(ids.numel() + 1, s["D"], dtype=torch.float64, device="cuda")
        torch.cumsum(s["dy"][order].double(), 0, out=sums[1:])
        upto = sums[run_ends]
        upto[1:] -= upto[:-1].clone()
        return upto * s["scale"]
    total = math.sqrt(math.fsum(float(torch.linalg.vector_norm(g.double().flatten()) ** 2) for g in s["grads"]))
    factor = min(1.0, 1.0 / (total + 1e-6))
    return {"norm": torch.tensor([total], dtype=torch.float64), "grads": [g.double() * factor for g in s["grads"]]}


def _exact_ce(s):
    """log sum exp of the products, minus the target's; the gradient sum over the words of
    (softmax - [word is the target]) times the row's weight, in pieces of 8192 words."""
    h, w, t = s["h"].double(), s["w"], s["t"].long()
    T, V = h.shape[0], w.shape[0]
    live = (t >= 0) & (t < V)
    parts = [torch.logsumexp(h @ w[v:v + 8192].double().T, dim=1) for v in range(0, V, 8192)]
    lse = torch.logsumexp(torch.stack(parts), dim=0)
    loss = torch.zeros_like(lse)
    loss[live] = lse[live] - (h[live] * w[t[live]].double()).sum(dim=1)
    if not s["grad"]:
        return {"loss": loss, "lse": lse}
    share = s["weight"].double() if s["weight"] is not None else torch.full_like(lse, 1.0 / max(1, int(live.sum())))
    share = share * live
    dh = torch.zeros_like(h)
    dw = torch.zeros(w.shape, dtype=torch.float64, device="cuda")
    for v in range(0, V, 8192):
        piece = w[v:v + 8192].double()
        d = torch.exp(h @ piece.T - lse[:, None])
        mine = live & (t >= v) & (t < v + piece.shape[0])
        d[mine, t[mine] - v] -= 1.0
        d *= share[:, None]
        dh += d @ piece
        dw[v:v + 8192] = d.T @ h
    return {"loss": loss, "dh": dh, "dw": dw}
