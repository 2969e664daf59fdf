"""Gradients of rows that see few keys, where ds = p (do.v - delta) is a small difference: delta is taken
from the weights and do.v, not from the rounded out, so dq and dk keep the precision of their own
roundings.

Bounds: as in window_ref, without the rounding of out: with f = (d_v + 8) 2^-24 sum|do||v| for an fp32
dot product over the values and e the relative error of a weight (2 e_s of window_ref), delta's average
of do.v is off by at most max f + e max|do.v - delta| over the row's keys, so
  |ds' - ds| <= p (f + max f + e max|do.v - delta|) + |ds| (H + e),   H = 2^-8 the rounding to bf16,
and dq, dk add their own H."""
import pytest
import torch

from dynamic_block_sparse_scoring_b200 import abi
from tests.window_ref import H, check, visible, window_ref

pytestmark = pytest.mark.gpu


def few_keys_ref(q, k, v, vis, scale, d_out):
    """{dq, dk: (value, bound)} with the bounds of the head comment."""
    B, Tq, Hq, d = q.shape
    Hkv, Tk, dv = k.shape[1], k.shape[2], v.shape[-1]
    G = Hq // Hkv
    q, k, v, do = q.double(), k.double(), v.double(), d_out.double()
    kk, vv = k.repeat_interleave(G, 1), v.repeat_interleave(G, 1)
    s = (torch.einsum("bthd,bhud->bhtu", q, kk) * scale).masked_fill(~vis, -torch.inf)
    p = torch.softmax(s, -1)
    dp = torch.einsum("bthd,bhud->bhtu", do, vv)
    delta = (p * dp).sum(-1, keepdim=True)
    ds = p * (dp - delta)
    qk = torch.einsum("bthd,bhud->bhtu", q.abs(), kk.abs()).masked_fill(~vis, 0).amax(-1, keepdim=True)
    e = 2 * ((d + 8) * 2.0 ** -24 * scale * qk + 2.0 ** -20)
    f = (dv + 8) * 2.0 ** -24 * torch.einsum("bthd,bhud->bhtu", do.abs(), vv.abs()).masked_fill(~vis, 0)
    far = (dp - delta).abs().masked_fill(~vis, 0).amax(-1, keepdim=True)
    err = p * (f + f.amax(-1, keepdim=True) + e * far) + ds.abs() * (H + e)
    fold = lambda x: x.view(B, Hkv, G, Tk, -1).sum(2)  # noqa: E731
    out = {"dq": (torch.einsum("bhtu,bhud->bthd", ds, kk), torch.einsum("bhtu,bhud->bthd", err, kk.abs())),
           "dk": (fold(torch.einsum("bhtu,bthd->bhud", ds, q)), fold(torch.einsum("bhtu,bthd->bhud", err, q.abs())))}
    return {n: (x * scale, b * scale + H * (x * scale).abs() + 1e-9) for n, (x, b) in out.items()}


# batch, Tq, q_pos0, h_q, h_kv, d_qk, d_v, window, sink
CASES = {
    "one_token": (2, 1, 0, 4, 2, 64, 64, 1, 0),
    "two_tokens": (3, 2, 0, 4, 1, 128, 128, 5, 0),
    "one_token_late": (2, 1, 300, 8, 1, 192, 128, 2, 0),
    "window_2": (1, 300, 0, 8, 2, 128, 128, 2, 0),
    "window_3_sinks": (2, 170, 40, 6, 2, 64, 128, 3, 2),
    "window_16_mha": (1, 400, 0, 3, 3, 128, 64, 16, 1),
    "window_50_sinks_9": (1, 333, 0, 16, 1, 192, 128, 50, 9),
    "sinks_40": (1, 260, 90, 5, 1, 128, 128, 2, 40),
    "group_33": (1, 90, 0, 33, 1, 64, 64, 20, 0),
    "group_64": (1, 70, 3, 64, 1, 192, 64, 8, 3),
    "many_planes": (2, 200, 0, 76, 76, 64, 64, 7, 0),
    "d256": (1, 90, 0, 4, 2, 256, 256, 4, 1),
    "group_72": (1, 50, 7, 72, 1, 64, 64, 3, 2),
}


def _make(name, seed):
    B, T, q0, Hq, Hkv, dqk, dv, W, ns = CASES[name]
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    r = lambda *s: torch.randn(*s, generator=g, device="cuda").to(torch.bfloat16)  # noqa: E731
    cfg = abi.window_config(B, T, q0 + T, Hq, Hkv, dqk, dv, W, ns, q0)
    return cfg, r(B, T, Hq, dqk), r(B, Hkv, q0 + T, dqk), r(B, Hkv, q0 + T, dv), r(B, T, Hq, dv), \
        visible(T, q0 + T, q0, W, ns, "cuda")


@pytest.mark.parametrize("name", sorted(CASES))
def test_gradients_of_few_keys(name):
    cfg, q, k, v, d_out, vis = _make(name, 41)
    assert int(vis.sum(1).max()) <= 64
    out, lse = abi.window_forward(cfg, q, k, v)
    dq, dk, dvv = abi.window_backward(cfg, q, k, v, out, lse, d_out)
    assert abi.nsa_get_device_status() == 0
    ref = few_keys_ref(q, k, v, vis, cfg.scale, d_out)
    check(dq, ref["dq"], f"{name} dq")
    check(dk, ref["dk"], f"{name} dk")
    check(dvv, window_ref(q, k, v, vis, cfg.scale, d_out)["dv"], f"{name} dv")


def test_rows_with_few_and_with_many_keys_in_one_call():
    """Full causal attention: the first query tiles are walked twice, the others once, several to a CTA;
    repeated calls give the same bits."""
    B, T, Hq, Hkv, dqk, dv = 4, 700, 12, 6, 192, 128
    g = torch.Generator(device="cuda")
    g.manual_seed(42)
    r = lambda *s: torch.randn(*s, generator=g, device="cuda").to(torch.bfloat16)  # noqa: E731
    q, k, v, d_out = r(B, T, Hq, dqk), r(B, Hkv, T, dqk), r(B, Hkv, T, dv), r(B, T, Hq, dv)
    cfg = abi.window_config(B, T, T, Hq, Hkv, dqk, dv, T, 0)
    out, lse = abi.window_forward(cfg, q, k, v)
    grads = abi.window_backward(cfg, q, k, v, out, lse, d_out)
    for _ in range(10):
        for a, b in zip(grads, abi.window_backward(cfg, q, k, v, out, lse, d_out)):
            assert torch.equal(a, b)
    vis = visible(T, T, 0, T, 0, "cuda")
    ref = window_ref(q, k, v, vis, cfg.scale, d_out)
    for n, x in zip(("dq", "dk", "dv"), grads):
        check(x, ref[n], n)
    sharp = few_keys_ref(q, k, v, vis, cfg.scale, d_out)["dq"]
    check(grads[0][:, :64], (sharp[0][:, :64], sharp[1][:, :64]), "dq of the first rows")
