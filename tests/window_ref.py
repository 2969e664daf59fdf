"""Sliding-window attention with sink tokens from its definition, in 64 bits, with the bounds that
the library's roundings allow.

vis(t) = {u <= t : u > t - window or u < sink};  s = scale q.k;  p = softmax over vis(t);
o = p v;  ds = p (do.v - do.o);  dq = scale ds k;  dk = scale ds^T q;  dv = p^T do.

Bounds (H = 2^-8, half a bf16 step relative to the value):
* the kernels round the weights p (and ds) to bf16 before the product that uses them and the
  result once more, so |o' - o| <= H sum p|v| + H|o|, and likewise for the gradients;
* the backward's delta = do.o reads the rounded o, so ds is off by p sum_c |do_c| |o'_c - o_c|;
* scores, exponentials and sums are fp32: a score is off by at most e_s = (d + 8) 2^-24 scale
  sum|q||k|, which moves p by a factor 1 +- 2 e_s (its own and the normaliser's), lse by e_s;
  ex2.approx and the fp32 sums add below 2^-20 of the value.
"""
import math

import torch

H = 2.0 ** -8


def visible(Tq, Tk, q0, window, sink, device):
    t = q0 + torch.arange(Tq, device=device).unsqueeze(1)
    u = torch.arange(Tk, device=device).unsqueeze(0)
    return (u <= t) & ((u > t - window) | (u < sink))


def window_ref(q, k, v, vis, scale, d_out=None):
    """q [B, Tq, Hq, d], k / v [B, Hkv, Tk, d] in any type; vis [Tq, Tk] or [B, Tq, Tk].

    Returns {name: (value, bound)} for out and lse, and dq, dk, dv when d_out is given; rows
    without a visible key have out = 0 and lse = -inf.
    """
    B, Tq, Hq, d = q.shape
    Hkv, Tk = k.shape[1], k.shape[2]
    G = Hq // Hkv
    q, k, v = q.double(), k.double(), v.double()
    kk, vv = k.repeat_interleave(G, 1), v.repeat_interleave(G, 1)              # [B, Hq, Tk, d]
    vis = (vis if vis.dim() == 3 else vis.unsqueeze(0).expand(B, -1, -1)).unsqueeze(1)
    s = torch.einsum("bthd,bhud->bhtu", q, kk) * scale
    s = s.masked_fill(~vis, -math.inf)
    m = s.amax(-1, keepdim=True).clamp(min=-1e300)
    e = torch.exp(s - m)
    z = e.sum(-1, keepdim=True)
    p = e / z.clamp(min=1e-300)
    lse = torch.where(z > 0, m + z.log(), torch.full_like(z, -math.inf)).squeeze(-1)
    o = torch.einsum("bhtu,bhud->bthd", p, vv)
    qk = torch.einsum("bthd,bhud->bhtu", q.abs(), kk.abs()).masked_fill(~vis, 0).amax(-1, keepdim=True)
    es = (d + 8) * 2.0 ** -24 * scale * qk + 2.0 ** -20                       # [B, Hq, Tq, 1]
    pv = torch.einsum("bhtu,bhud->bthd", p * (H + 2 * es), vv.abs())
    o_bound = pv + H * o.abs() + 1e-6
    out = {"out": (o, o_bound),
           "lse": (lse.transpose(1, 2),
                   (es.squeeze(-1) + 2.0 ** -20 * lse.abs().clamp(max=1e30)).transpose(1, 2) + 1e-6)}
    if d_out is None:
        return out
    do = d_out.double()
    delta = (do * o).sum(-1).transpose(1, 2).unsqueeze(-1)                     # [B, Hq, Tq, 1]
    dp = torch.einsum("bthd,bhud->bhtu", do, vv)
    ds = p * (dp - delta)
    fold = lambda x: x.view(B, Hkv, G, Tk, -1).sum(2)  # noqa: E731
    out["dq"] = torch.einsum("bhtu,bhud->bthd", ds, kk) * scale
    out["dk"] = fold(torch.einsum("bhtu,bthd->bhud", ds, q)) * scale
    out["dv"] = fold(torch.einsum("bhtu,bthd->bhud", p, do))
    d_delta = (do.abs() * o_bound).sum(-1).transpose(1, 2).unsqueeze(-1)
    fp = (v.shape[-1] + 8) * 2.0 ** -24 * torch.einsum("bthd,bhud->bhtu", do.abs(), vv.abs())
    ds_err = p * (d_delta + fp) + ds.abs() * (H + 2 * es)
    p_err = p * (H + 2 * es)
    bound = {"dq": torch.einsum("bhtu,bhud->bthd", ds_err, kk.abs()) * scale,
             "dk": fold(torch.einsum("bhtu,bthd->bhud", ds_err, q.abs())) * scale,
             "dv": fold(torch.einsum("bhtu,bthd->bhud", p_err, do.abs()))}
    for n in ("dq", "dk", "dv"):
        out[n] = (out[n], bound[n] + H * out[n].abs() + 1e-6)
    return out


def check(got, want, what):
    """got: tensor; want: (value, bound)."""
    value, bound = want
    g = got.double()
    assert g.shape == value.shape, what
    inf = torch.isinf(value)
    assert torch.equal(g[inf], value[inf]), f"{what}: infinities differ"
    err = torch.where(inf, torch.zeros_like(g), (g - value).abs())
    bad = ~(err <= bound)
    assert not bad.any(), (f"{what}: {int(bad.sum())} of {bad.numel()} values over the bound, worst "
                           f"{float((err / bound)[bad].max()):.3g} times it, first at "
                           f"{bad.nonzero()[0].tolist()}")
