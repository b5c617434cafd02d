"""Attention and its gradient from the definitions in 64 bits, with a bound per entry on
what the kernels' roundings may add up to.

The bounds.  Scores are FP32 sums of D exact products: their error is at most
(D + 4) U A, A = scale * sum |q||k| (one rounding per term, a few for the scale), U = 2^-23 (a
step, so that sums which truncate are covered).  p = exp(s - lse) takes the score's and lse's:
rel = exp(2 (D + 4) U A + n U) - 1 with n terms in the sum.  p enters the product with v rounded to
BF16 (u = 2^-8) and the result is rounded once:
  out: (u + rel + n U) sum p |v| + u |out|.
delta is the sum of dout and the rounded out: its error is sum |dout| (bound of out) + D U sum |dout||out|.
ds = p (dp - delta), rounded to BF16, then multiplied and summed:
  dq: scale sum (u |ds| + p (rel |dp - delta| + error of delta + D U sum |dout||v|)) |k| + n U .. + u |dq|,
dk likewise over the queries, dv as out.
FP32 and BF16 values below 2^-126 have lost bits or are zero: p, ds, a term and a result may each
be off by TINY = 2^-126 besides (scores that differ by more than 87 leave such p)."""
import torch

U, HALF, TINY = 2.0 ** -23, 2.0 ** -8, 2.0 ** -126


def seen_mask(nq, nk, causal, window, device="cpu"):
    i = torch.arange(nq, device=device).unsqueeze(1) + (nk - nq)
    j = torch.arange(nk, device=device)
    m = torch.ones(nq, nk, dtype=torch.bool, device=device)
    if causal:
        m &= j <= i
        if window:
            m &= j > i - window
    return m


def _tiny(seen, x):
    return TINY * (2 + seen.double() @ (1 + x.abs()))


def head(q, k, v, seen, scale, dout=None):
    """Float64 (out, lse, dq, dk, dv) of one head and the bounds of each; q [nq][D], k, v
    [nk][D] float64, seen [nq][nk].  What is not seen is not touched, whatever it holds."""
    D, n = q.shape[1], k.shape[0]
    zero = torch.zeros((), dtype=torch.float64, device=q.device)
    z = torch.where(seen, scale * (q @ k.T), zero)
    mag = torch.where(seen, scale * (q.abs() @ k.abs().T), zero)
    top = torch.where(seen, z, -torch.inf).max(1, keepdim=True).values if n else z.new_zeros(z.shape[0], 1)
    any_ = seen.any(1, keepdim=True)
    top = torch.where(any_, top, zero)
    e = torch.where(seen, torch.exp(z - top), zero)
    total = e.sum(1, keepdim=True)
    p = torch.where(any_, e / torch.where(any_, total, zero + 1), zero)
    lse = torch.where(any_, top + torch.log(total), zero - torch.inf).squeeze(1)
    count = seen.sum(1, keepdim=True).double()
    most = mag.max(1, keepdim=True).values if n else mag.new_zeros(mag.shape[0], 1)
    s_err = (D + 4) * U * most
    rel = torch.exp(2 * s_err + count * U) - 1
    out = p @ v
    out_tol = (HALF + rel + count * U) * (p @ v.abs()) + HALF * out.abs() + _tiny(seen, v)
    lse_tol = (s_err + count * U + U * (1 + torch.where(any_, lse.unsqueeze(1).abs(), zero) + most)).squeeze(1)
    res = {"out": out, "lse": lse}
    tol = {"out": out_tol, "lse": lse_tol}
    if dout is None:
        return res, tol
    nq = q.shape[0]
    dp = dout @ v.T
    delta = (dout * out).sum(1, keepdim=True)
    d_err = (dout.abs() * out_tol).sum(1, keepdim=True) + D * U * (dout * out).abs().sum(1, keepdim=True)
    dp_err = D * U * (dout.abs() @ v.abs().T)
    ds = p * (dp - delta)
    ds_err = (HALF + U) * ds.abs() + (1 + HALF) * p * (rel * (dp - delta).abs() + d_err + dp_err)
    ds_err = ds_err + TINY * seen * (2 + (dp - delta).abs())
    res["dq"], res["dk"], res["dv"] = scale * (ds @ k), scale * (ds.T @ q), p.T @ dout
    tol["dq"] = scale * ((ds_err + n * U * ds.abs()) @ k.abs()) + HALF * res["dq"].abs() \
        + _tiny(seen, k)
    tol["dk"] = scale * ((ds_err + nq * U * ds.abs()).T @ q.abs()) + _tiny(seen.T, q)
    tol["dv"] = ((HALF + rel + nq * U) * p).T @ dout.abs() + _tiny(seen.T, dout)
    return res, tol


def attention(q, k, v, scale, causal, window, bounds=None, dout=None):
    """All heads.  q [B][T][H][D], or [T][H][D] with bounds = the (q0, q1, k0, k1) of each
    sequence.  Returns (results, bounds) as float64 of the operands' shapes; rows outside every
    sequence are zeros (lse -inf) and exact."""
    q, k, v = q.double(), k.double(), v.double()
    dout = None if dout is None else dout.double()
    names = ("out", "lse") if dout is None else ("out", "lse", "dq", "dk", "dv")
    like = {"out": q, "lse": q[..., 0], "dq": q, "dk": k, "dv": v}
    res = {n: torch.zeros_like(like[n]) for n in names}
    tol = {n: torch.zeros_like(like[n]) for n in names}
    res["lse"].fill_(-torch.inf)
    G = q.shape[-2] // k.shape[-2]
    if bounds is None:
        if q.dim() == 3:
            places = [(slice(0, q.shape[0]), slice(0, k.shape[0]))]
        else:
            places = [(b, b) for b in range(q.shape[0])]
    else:
        places = [(slice(a, b), slice(c, d)) for a, b, c, d in bounds]
    for iq, ik in places:
        seen = seen_mask(q[iq].shape[0], k[ik].shape[0], causal, window, q.device)
        for h in range(q.shape[-2]):
            r, t = head(q[iq][:, h], k[ik][:, h // G], v[ik][:, h // G], seen, scale,
                        None if dout is None else dout[iq][:, h])
            for n in names:
                if n in ("dk", "dv"):
                    res[n][ik][:, h // G] += r[n]
                    tol[n][ik][:, h // G] += t[n]
                else:
                    res[n][iq][:, h] = r[n]
                    tol[n][iq][:, h] = t[n]
    for n in ("dk", "dv"):   # the sum over a group's heads is rounded once
        if n in res:
            tol[n] += HALF * res[n].abs()
    return res, tol
