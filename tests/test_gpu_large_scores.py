"""Scaled scores far beyond the usual range: |scale q.k| up to 1e32.  The scores q.k here are whole
numbers that fp32 holds exactly, so the softmax has a sharp value at any scale: the keys of the row's
largest score share the weight, or, where scores differ by a few units after scaling, the weights
depend on exact differences.

Bounds (H = 2^-8, half a bf16 step): the weights enter the value product as bf16 and the result is
rounded once more, |o' - o| <= 2 H sum p|v|; fp32 sums and ex2 add below 2^-16 of that.  lse is a
product and a sum in fp32 with constants of 24 bits, 8 roundings: below 2^-20 |lse|."""
import math

import pytest
import torch

from dynamic_block_sparse_scoring_b200 import abi
from tests.paged_ref import filled
from tests.window_ref import check, visible, window_ref

pytestmark = pytest.mark.gpu

H = 2.0 ** -8


def _bounded(ref, q, k, v, vis, scale):
    """window_ref's out and lse with the bounds of the head comment."""
    B, Tq, Hq, _ = q.shape
    G = Hq // k.shape[1]
    ones = window_ref(q, k, v.abs(), vis, scale)["out"][0]                     # sum p|v|
    out, lse = ref["out"][0], ref["lse"][0]
    return {"out": (out, (2 * H + 2.0 ** -16) * ones + 1e-6), "lse": (lse, 2.0 ** -20 * lse.abs() + 1e-6)}


def _whole(g, lo, hi, *shape):
    return torch.randint(lo, hi + 1, shape, generator=g, device="cuda").to(torch.bfloat16)


# Tq, q_pos0, h_q, h_kv, d_qk, d_v, window, sink
SHAPES = {
    "singles": (300, 0, 4, 2, 64, 64, 1000, 0),
    "window_sinks": (257, 90, 6, 2, 128, 128, 130, 70),
    "short_window": (140, 0, 3, 1, 192, 128, 2, 0),
    "pairs": (300, 0, 152, 152, 64, 64, 140, 3),
    "ffma_256": (70, 5, 4, 2, 256, 256, 30, 2),
    "ffma_group_72": (40, 0, 72, 1, 64, 64, 20, 3),
}


@pytest.mark.parametrize("scale", [1e6, 1e9, 1e30])
@pytest.mark.parametrize("name", sorted(SHAPES))
def test_forward_gives_the_weight_to_the_largest_scores(name, scale):
    """Scores of -60 to 60 with many ties, positive and negative maxima, maxima that move between tiles."""
    T, q0, Hq, Hkv, dqk, dv, W, ns = SHAPES[name]
    g = torch.Generator(device="cuda")
    g.manual_seed(21)
    q, k = _whole(g, -1, 1, 1, T, Hq, dqk), _whole(g, -1, 1, 1, Hkv, q0 + T, dqk)
    v = torch.randn(1, Hkv, q0 + T, dv, generator=g, device="cuda").to(torch.bfloat16)
    cfg = abi.window_config(1, T, q0 + T, Hq, Hkv, dqk, dv, W, ns, q0, scale=scale)
    out, lse = abi.window_forward(cfg, q, k, v)
    assert torch.isfinite(out).all() and torch.isfinite(lse).all()
    vis = visible(T, q0 + T, q0, W, ns, "cuda")
    ref = _bounded(window_ref(q, k, v, vis, cfg.scale), q, k, v, vis, cfg.scale)
    check(out, ref["out"], f"{name} out")
    check(lse, ref["lse"], f"{name} lse")


@pytest.mark.parametrize("name", ["singles", "window_sinks", "pairs"])
def test_small_differences_of_scores_around_2_to_the_24(name):
    """Scaled scores 2^24 + 2 j in units of log 2, |j| <= 20: the weights are 2^(2 (j - j')), on either
    side of the size from which the reference is subtracted first, and the reference moves from one
    side to the other."""
    T, q0, Hq, Hkv, dqk, dv, W, ns = SHAPES[name]
    g = torch.Generator(device="cuda")
    g.manual_seed(22)
    q = torch.zeros(1, T, Hq, dqk, dtype=torch.bfloat16, device="cuda")
    k = torch.zeros(1, Hkv, q0 + T, dqk, dtype=torch.bfloat16, device="cuda")
    q[..., 0], q[..., 1], k[..., 0] = 2048, 1, 4096
    k[..., 1] = _whole(g, -20, 20, 1, Hkv, q0 + T)
    k[..., : (q0 + T) // 3, 1] = -20                 # the first third stays below: the maximum moves
    v = torch.randn(1, Hkv, q0 + T, dv, generator=g, device="cuda").to(torch.bfloat16)
    cfg = abi.window_config(1, T, q0 + T, Hq, Hkv, dqk, dv, W, ns, q0, scale=2 * math.log(2))
    out, lse = abi.window_forward(cfg, q, k, v)
    vis = visible(T, q0 + T, q0, W, ns, "cuda")
    ref = _bounded(window_ref(q, k, v, vis, cfg.scale), q, k, v, vis, cfg.scale)
    check(out, ref["out"], f"{name} out")
    check(lse, ref["lse"], f"{name} lse")


@pytest.mark.parametrize("scale", [1e6, 1e9, 1e30])
@pytest.mark.parametrize("dims", [(4, 2, 64, 64), (4, 2, 192, 128), (4, 2, 256, 256), (72, 1, 64, 64)], ids=str)
def test_backward_weights_stay_below_one(dims, scale):
    """Every key has a score of its own, so one key has each row's whole weight: dv is the sum of the
    d_out of the rows whose largest score the key is; dq and dk are 0 but for scale times fp32's noise."""
    Hq, Hkv, dqk, dv = dims
    T = 200
    g = torch.Generator(device="cuda")
    g.manual_seed(23)
    k = torch.randn(1, Hkv, T, dqk, generator=g, device="cuda").to(torch.bfloat16)
    for h in range(Hkv):
        k[0, h, :, 0] = (torch.randperm(T, generator=g, device="cuda") - T // 2).to(torch.bfloat16)
    q = torch.zeros(1, T, Hq, dqk, dtype=torch.bfloat16, device="cuda")
    q[..., 0] = torch.where(_whole(g, 0, 1, 1, T, Hq) > 0, 2.0, -3.0)
    r = lambda *s: torch.randn(*s, generator=g, device="cuda").to(torch.bfloat16)  # noqa: E731
    v, d_out = r(1, Hkv, T, dv), r(1, T, Hq, dv)
    cfg = abi.window_config(1, T, T, Hq, Hkv, dqk, dv, 90, 7, scale=scale)
    out, lse = abi.window_forward(cfg, q, k, v)
    got = abi.window_backward(cfg, q, k, v, out, lse, d_out)
    for x in got:
        assert torch.isfinite(x).all()
    vis = visible(T, T, 0, 90, 7, "cuda")
    ref = window_ref(q, k, v, vis, cfg.scale, d_out)["dv"][0]
    size = window_ref(q, k, v, vis, cfg.scale, d_out.abs())["dv"][0]           # sum p|d_out|
    check(got[2], (ref, (2 * H + 2.0 ** -16) * size + 1e-6), "dv")



@pytest.mark.parametrize("dims", [(6, 2, 128, 128), (160, 160, 64, 64), (4, 2, 256, 256)], ids=str)
@pytest.mark.parametrize("large", [(5,), (0, 3, 130, 299)])
def test_a_few_rows_with_large_scores_among_ordinary_ones(large, dims):
    """Queries `large` are 2^20 times a unit vector whose scores are whole numbers (one key has all the
    weight), the others have none of that column; dv holds both, dq of the ordinary rows and the other
    columns of dk are as without the large rows."""
    Hq, Hkv, dqk, dv = dims
    T, W, ns = 300, 90, 7
    g = torch.Generator(device="cuda")
    g.manual_seed(25)
    r = lambda *s: torch.randn(*s, generator=g, device="cuda").to(torch.bfloat16)  # noqa: E731
    q, k, v, d_out = r(1, T, Hq, dqk), r(1, Hkv, T, dqk), r(1, Hkv, T, dv), r(1, T, Hq, dv)
    q[..., 0] = 0
    q[:, large] = 0
    q[:, large, :, 0] = 2.0 ** 20
    for h in range(Hkv):
        k[0, h, :, 0] = (torch.randperm(T, generator=g, device="cuda") - T // 2).to(torch.bfloat16)
    cfg = abi.window_config(1, T, T, Hq, Hkv, dqk, dv, W, ns)
    out, lse = abi.window_forward(cfg, q, k, v)
    dq, dk, dvv = abi.window_backward(cfg, q, k, v, out, lse, d_out)
    vis = visible(T, T, 0, W, ns, "cuda")
    some = torch.zeros_like(d_out)
    some[:, large] = d_out[:, large]
    ref = window_ref(q, k, v, vis, cfg.scale, d_out - some)
    part = window_ref(q, k, v, vis, cfg.scale, some)["dv"][0]
    size = window_ref(q, k, v, vis, cfg.scale, some.abs())["dv"][0]
    check(dvv, (ref["dv"][0] + part, ref["dv"][1] + (2 * H + 2.0 ** -16) * size), "dv")
    rest = [t for t in range(T) if t not in large]
    check(dq[:, rest], (ref["dq"][0][:, rest], ref["dq"][1][:, rest]), "dq")
    check(dk[..., 1:], (ref["dk"][0][..., 1:], ref["dk"][1][..., 1:]), "dk")


@pytest.mark.parametrize("scale", [1e6, 1e9, 1e30])
@pytest.mark.parametrize("new, page, lens", [(1, 16, [700, 3, 64]), (3, 64, [2100])])
def test_paged_attention_gives_the_weight_to_the_largest_scores(scale, new, page, lens):
    cols = -(-max(lens) // page) + 1
    c = filled(len(lens), cols, sum(-(-n // page) for n in lens) + 2, page, 2, 128, 128, lens, 24)
    g = torch.Generator(device="cuda")
    g.manual_seed(24)
    c.k = torch.where(c.k.isnan(), c.k, c.k.float().round().clamp(-1, 1).to(torch.bfloat16))
    x = c.on_gpu()
    q = _whole(g, -1, 1, len(lens), new, 8, 128)
    cfg = abi.paged_config(len(lens), new, 8, 2, 128, 128, page, len(c.ref), cols, scale=scale)
    out, lse = abi.paged_attention(cfg, q, x["k_pages"], x["v_pages"], x["table"], x["lens"])
    assert torch.isfinite(out).all() and torch.isfinite(lse).all()
    for b, n in enumerate(lens):
        k, v = (y.unsqueeze(0).cuda() for y in c.dense(b))
        vis = visible(new, n, n - new, 1 << 30, 0, "cuda")
        ref = _bounded(window_ref(q[b:b + 1], k, v, vis, cfg.scale), q[b:b + 1], k, v, vis, cfg.scale)
        check(out[b:b + 1], ref["out"], f"row {b} out")
        check(lse[b:b + 1], ref["lse"], f"row {b} lse")
