"""Window attention with sink tokens (nsa_window_attn_fwd / _bwd) against the 64-bit definition."""
import pytest
import torch

from dynamic_block_sparse_scoring_b200 import abi
from tests.window_ref import check, visible, window_ref

pytestmark = pytest.mark.gpu

# batch, Tq, Tk - Tq - pos0 rows behind, q_pos0, h_q, h_kv, d_qk, d_v, window, sink
CASES = {
    "one_token": (1, 1, 0, 0, 4, 1, 64, 64, 1, 0),
    "one_token_late": (2, 1, 0, 300, 16, 2, 128, 128, 100, 3),
    "two_tokens_window_1": (1, 2, 0, 0, 2, 2, 64, 128, 1, 0),
    "window_1_sinks": (1, 70, 0, 0, 4, 2, 128, 64, 1, 5),
    "tiny": (1, 333, 0, 0, 4, 1, 64, 64, 128, 4),
    "gqa16_192": (1, 200, 0, 0, 32, 2, 192, 128, 50, 7),
    "mha": (2, 300, 0, 0, 3, 3, 128, 128, 130, 16),
    "group_3": (1, 190, 0, 0, 6, 2, 128, 128, 64, 1),
    "group_6": (1, 150, 0, 0, 12, 2, 192, 128, 64, 70),
    "group_12_192_64": (1, 129, 0, 0, 12, 1, 192, 64, 40, 2),
    "group_64": (1, 67, 0, 0, 64, 1, 128, 128, 20, 3),
    "group_72": (1, 40, 0, 0, 72, 1, 64, 64, 20, 3),
    "full_causal": (1, 400, 0, 0, 4, 2, 128, 128, 400, 0),
    "window_over_cache": (1, 257, 0, 0, 4, 4, 64, 64, 100000, 9),
    "all_sinks": (1, 260, 0, 0, 4, 2, 128, 128, 3, 1000),
    "sinks_meet_window": (1, 300, 0, 0, 4, 2, 128, 128, 64, 65),
    "long_window_edges": (1, 513, 0, 0, 2, 1, 128, 128, 128, 128),
    "chunk": (2, 100, 0, 411, 8, 2, 192, 128, 150, 20),
    "chunk_rows_behind": (2, 90, 77, 300, 8, 2, 128, 128, 128, 10),
    "d256": (1, 90, 0, 0, 4, 2, 256, 256, 33, 4),
    "d256_v64": (2, 61, 5, 40, 2, 1, 256, 64, 30, 4),
    "many_key_tiles": (1, 1500, 0, 0, 8, 1, 64, 64, 700, 40),
}


def make(name, seed=0, spread=1.0):
    B, Tq, behind, q0, Hq, Hkv, dqk, dv, W, ns = CASES[name]
    Tk = q0 + Tq + behind
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    r = lambda *s: (torch.randn(*s, generator=g, device="cuda") * spread).to(torch.bfloat16)  # noqa: E731
    cfg = abi.window_config(B, Tq, Tk, Hq, Hkv, dqk, dv, W, ns, q0)
    x = dict(q=r(B, Tq, Hq, dqk), k=r(B, Hkv, Tk, dqk), v=r(B, Hkv, Tk, dv))
    return cfg, x, r(B, Tq, Hq, dv), visible(Tq, Tk, q0, W, ns, "cuda")


@pytest.mark.parametrize("name", sorted(CASES))
def test_forward_and_backward(name):
    cfg, x, d_out, vis = make(name)
    out, lse = abi.window_forward(cfg, **x)
    dq, dk, dv = abi.window_backward(cfg, **x, out=out, lse=lse, d_out=d_out)
    torch.cuda.synchronize()
    assert abi.nsa_get_device_status() == 0
    ref = window_ref(x["q"], x["k"], x["v"], vis, cfg.scale, d_out)
    for n, got in [("out", out), ("lse", lse), ("dq", dq), ("dk", dk), ("dv", dv)]:
        check(got, ref[n], f"{name} {n}")


@pytest.mark.parametrize("name", ["tiny", "gqa16_192", "sinks_meet_window"])
def test_large_scores(name):
    """Scores of several hundred: the running maximum moves often, weights underflow."""
    cfg, x, d_out, vis = make(name, seed=1, spread=6.0)
    out, lse = abi.window_forward(cfg, **x)
    grads = abi.window_backward(cfg, **x, out=out, lse=lse, d_out=d_out)
    ref = window_ref(x["q"], x["k"], x["v"], vis, cfg.scale, d_out)
    for n, got in zip(("out", "lse", "dq", "dk", "dv"), (out, lse) + grads):
        check(got, ref[n], f"{name} {n}")


@pytest.mark.parametrize("scale", [1e-30, 1e-3, 3.0])
def test_other_scales(scale):
    """A scale so small that every weight is equal, and one that makes the softmax sharp; 21 tokens of
    three heads leave rows of the streamed tiles without a query."""
    g = torch.Generator(device="cuda")
    g.manual_seed(8)
    r = lambda *s: torch.randn(*s, generator=g, device="cuda").to(torch.bfloat16)  # noqa: E731
    q, k, v, d_out = r(1, 85, 6, 64), r(1, 2, 85, 64), r(1, 2, 85, 64), r(1, 85, 6, 64)
    cfg = abi.window_config(1, 85, 85, 6, 2, 64, 64, 30, 3, scale=scale)
    out, lse = abi.window_forward(cfg, q, k, v)
    grads = abi.window_backward(cfg, q, k, v, out, lse, d_out)
    ref = window_ref(q, k, v, visible(85, 85, 0, 30, 3, "cuda"), cfg.scale, d_out)
    for n, got in zip(("out", "lse", "dq", "dk", "dv"), (out, lse) + grads):
        check(got, ref[n], n)


@pytest.mark.parametrize("group", [1, 5, 33])
@pytest.mark.parametrize("window", [1, 3, 90])
def test_short_windows_without_sinks(window, group):
    """No key tile holds sinks, and none of the others has enough queries to be cut into items."""
    Tq, q0 = 700, 37
    Tk = q0 + Tq
    g = torch.Generator(device="cuda")
    g.manual_seed(9)
    r = lambda *s: torch.randn(*s, generator=g, device="cuda").to(torch.bfloat16)  # noqa: E731
    q, k, v, d_out = r(1, Tq, group, 64), r(1, 1, Tk, 64), r(1, 1, Tk, 128), r(1, Tq, group, 128)
    cfg = abi.window_config(1, Tq, Tk, group, 1, 64, 128, window, 0, q0)
    out, lse = abi.window_forward(cfg, q, k, v)
    grads = abi.window_backward(cfg, q, k, v, out, lse, d_out)
    ref = window_ref(q, k, v, visible(Tq, Tk, q0, window, 0, "cuda"), cfg.scale, d_out)
    for n, got in zip(("out", "lse", "dq", "dk", "dv"), (out, lse) + grads):
        check(got, ref[n], n)


@pytest.mark.parametrize("window, sink", [(1, 0), (1, 3), (1, 300), (129, 150), (129, 128), (128, 257), (100, 129),
                                          (257, 400), (40, 1000), (1000, 7)])
@pytest.mark.parametrize("tokens, group, pos0", [(390, 1, 0), (131, 3, 256)])
def test_many_planes(tokens, group, pos0, window, sink):
    """152 (sequence, KV head) planes: work items of two query tiles whose windows and sinks need
    different key tiles."""
    Tk = pos0 + tokens
    g = torch.Generator(device="cuda")
    g.manual_seed(10)
    r = lambda *s: torch.randn(*s, generator=g, device="cuda").to(torch.bfloat16)  # noqa: E731
    q, k, v = r(2, tokens, 76 * group, 64), r(2, 76, Tk, 64), r(2, 76, Tk, 64)
    d_out = r(2, tokens, 76 * group, 64)
    cfg = abi.window_config(2, tokens, Tk, 76 * group, 76, 64, 64, window, sink, pos0)
    out, lse = abi.window_forward(cfg, q, k, v)
    grads = abi.window_backward(cfg, q, k, v, out, lse, d_out)
    ref = window_ref(q, k, v, visible(tokens, Tk, pos0, window, sink, "cuda"), cfg.scale, d_out)
    for n, got in zip(("out", "lse", "dq", "dk", "dv"), (out, lse) + grads):
        check(got, ref[n], n)


def test_lse_is_optional_and_calls_repeat_bit_for_bit():
    cfg, x, d_out, _ = make("gqa16_192", seed=2)
    out, lse = abi.window_forward(cfg, **x)
    bare = torch.empty_like(out)
    abi.nsa_window_attn_fwd(cfg, x["q"], x["k"], x["v"], bare)
    first = abi.window_backward(cfg, **x, out=out, lse=lse, d_out=d_out)
    second = abi.window_backward(cfg, **x, out=out, lse=lse, d_out=d_out)
    assert torch.equal(out, bare)
    for a, b in zip(first, second):
        assert torch.equal(a, b)


def test_no_queries():
    cfg = abi.window_config(2, 0, 50, 4, 2, 64, 64, 8)
    q = torch.empty(2, 0, 4, 64, dtype=torch.bfloat16, device="cuda")
    k = torch.randn(2, 2, 50, 64, device="cuda").to(torch.bfloat16)
    out, lse = abi.window_forward(cfg, q, k, k)
    dq, dk, dv = abi.window_backward(cfg, q, k, k, out, lse, out)
    assert out.shape == (2, 0, 4, 64) and dq.shape == q.shape and dk.shape == k.shape
    assert not dk.any() and not dv.any()


def test_a_padded_batch_leaves_its_sequences_alone():
    """Rows behind a sequence's end, with d_out = 0 there, change nothing before it."""
    cfg, x, d_out, _ = make("mha", seed=3)
    n = 211
    d_out[:, n:] = 0
    out, lse = abi.window_forward(cfg, **x)
    dq, dk, dv = abi.window_backward(cfg, **x, out=out, lse=lse, d_out=d_out)
    short = abi.window_config(2, n, n, 3, 3, 128, 128, 130, 16)
    y = dict(q=x["q"][:, :n].contiguous(), k=x["k"][:, :, :n].contiguous(), v=x["v"][:, :, :n].contiguous())
    vis = visible(n, n, 0, 130, 16, "cuda")
    ref = window_ref(y["q"], y["k"], y["v"], vis, short.scale, d_out[:, :n])
    check(out[:, :n], ref["out"], "out")
    check(dq[:, :n], ref["dq"], "dq")
    check(dk[:, :, :n], ref["dk"], "dk")
    check(dv[:, :, :n], ref["dv"], "dv")
    assert not dq[:, n:].any() and not dk[:, :, n:].any() and not dv[:, :, n:].any()


def test_captured_and_on_a_side_stream():
    cfg, x, d_out, vis = make("tiny", seed=4)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        out, lse = abi.window_forward(cfg, **x)
        abi.window_backward(cfg, **x, out=out, lse=lse, d_out=d_out)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        g_out, g_lse = abi.window_forward(cfg, **x)
        g_grads = abi.window_backward(cfg, **x, out=g_out, lse=g_lse, d_out=d_out)
    fresh = make("tiny", seed=5)
    for n in x:
        x[n].copy_(fresh[1][n])
    d_out.copy_(fresh[2])
    graph.replay()
    torch.cuda.synchronize()
    ref = window_ref(x["q"], x["k"], x["v"], vis, cfg.scale, d_out)
    for n, got in zip(("out", "lse", "dq", "dk", "dv"), (g_out, g_lse) + g_grads):
        check(got, ref[n], n)


def test_refuses_what_is_not_dense_or_of_another_type():
    cfg, x, _, _ = make("tiny")
    with pytest.raises(ValueError, match="contiguous"):
        abi.window_forward(cfg, x["q"].transpose(1, 2).contiguous().transpose(1, 2), x["k"], x["v"])
    with pytest.raises(ValueError, match="k is"):
        abi.window_forward(cfg, x["q"], x["k"].float(), x["v"])
    with pytest.raises(ValueError, match="one CUDA device"):
        abi.window_forward(cfg, x["q"], x["k"], x["v"].cpu())


@pytest.mark.parametrize("dims", [(192, 128), (128, 64), (64, 64)], ids=str)
def test_many_work_items_per_cta(dims):
    """Several work items on every CTA, forward and backward, some of them partial; twenty repetitions
    give the same bits (a hand-over between warps that is not waited for would show)."""
    dqk, dv = dims
    B, T, Hq, Hkv, W, ns = 2, 1210, 32, 8, 300, 70
    g = torch.Generator(device="cuda")
    g.manual_seed(9)
    r = lambda *s: torch.randn(*s, generator=g, device="cuda").to(torch.bfloat16)  # noqa: E731
    q, k, v, d_out = r(B, T, Hq, dqk), r(B, Hkv, T, dqk), r(B, Hkv, T, dv), r(B, T, Hq, dv)
    cfg = abi.window_config(B, T, T, Hq, Hkv, dqk, dv, W, ns)
    first = None
    for _ in range(20):
        out, lse = abi.window_forward(cfg, q, k, v)
        got = (out, lse) + abi.window_backward(cfg, q, k, v, out, lse, d_out)
        if first is None:
            first = got
        for a, b in zip(first, got):
            assert torch.equal(a, b)
    assert abi.nsa_get_device_status() == 0
    for b in range(B):
        ref = window_ref(q[b:b + 1], k[b:b + 1], v[b:b + 1], visible(T, T, 0, W, ns, "cuda"), cfg.scale,
                         d_out[b:b + 1])
        for n, x in zip(("out", "lse", "dq", "dk", "dv"), first):
            check(x[b:b + 1], ref[n], f"sequence {b} {n}")


def test_turned_steps_of_a_long_batch():
    """More query rows than the backward's natural order is kept for (64 MB of q and d_out), checked on
    the last of several sequences; key tiles with and without sinks, whole and cut."""
    B, T, Hq, Hkv, d, W, ns = 40, 900, 8, 1, 128, 200, 10
    g = torch.Generator(device="cuda")
    g.manual_seed(10)
    r = lambda *s: torch.randn(*s, generator=g, device="cuda").to(torch.bfloat16)  # noqa: E731
    q, k, v, d_out = r(B, T, Hq, d), r(B, Hkv, T, d), r(B, Hkv, T, d), r(B, T, Hq, d)
    assert B * T * Hq * 2 * d * 2 > 64 << 20
    cfg = abi.window_config(B, T, T, Hq, Hkv, d, d, W, ns)
    out, lse = abi.window_forward(cfg, q, k, v)
    grads = abi.window_backward(cfg, q, k, v, out, lse, d_out)
    for b in (0, B - 1):
        one = slice(b, b + 1)
        ref = window_ref(q[one], k[one], v[one], visible(T, T, 0, W, ns, "cuda"), cfg.scale, d_out[one])
        for n, x in zip(("out", "lse", "dq", "dk", "dv"), (out, lse) + grads):
            check(x[one], ref[n], f"sequence {b} {n}")


def test_offsets_past_32_bits():
    """Two planes of 9 million keys: the last tokens' keys lie past 2^31 elements."""
    Tk, Tq, d, W, ns = 9_000_000, 40, 128, 70, 3
    k = torch.zeros(1, 2, Tk, d, dtype=torch.bfloat16, device="cuda")
    v = torch.zeros_like(k)
    g = torch.Generator(device="cuda")
    g.manual_seed(12)
    r = lambda *s: torch.randn(*s, generator=g, device="cuda").to(torch.bfloat16)  # noqa: E731
    far = Tk - 200
    for x in (k, v):
        x[:, :, :ns], x[:, :, far:] = r(1, 2, ns, d), r(1, 2, 200, d)
    assert k.numel() > 1 << 31
    q, d_out = r(1, Tq, 4, d), r(1, Tq, 4, d)
    cfg = abi.window_config(1, Tq, Tk, 4, 2, d, d, W, ns, Tk - Tq)
    out, lse = abi.window_forward(cfg, q, k, v)
    dq, dk, dv = abi.window_backward(cfg, q, k, v, out, lse, d_out)
    near = lambda x: torch.cat([x[:, :, :ns], x[:, :, far:]], 2)  # noqa: E731
    vis = torch.cat([torch.ones(Tq, ns, dtype=torch.bool, device="cuda"),
                     visible(Tq, 200, 200 - Tq, W, 0, "cuda")], 1)
    ref = window_ref(q, near(k), near(v), vis, cfg.scale, d_out)
    for n, x in [("out", out), ("lse", lse), ("dq", dq), ("dk", near(dk)), ("dv", near(dv))]:
        check(x, ref[n], n)
    assert not dk[:, :, ns:far].any() and not dv[:, :, ns:far].any()


@pytest.mark.parametrize("dims", [(64, 64), (256, 256)], ids=str)
def test_a_query_that_is_not_a_number_shows_in_every_output(dims):
    """A NaN is not clamped away: its row's out, lse and dq and its keys' dk and dv are NaN."""
    dqk, dv = dims
    g = torch.Generator(device="cuda")
    g.manual_seed(14)
    r = lambda *s: torch.randn(*s, generator=g, device="cuda").to(torch.bfloat16)  # noqa: E731
    q, k, v, d_out = r(1, 90, 4, dqk), r(1, 2, 90, dqk), r(1, 2, 90, dv), r(1, 90, 4, dv)
    q[0, 50, 1, 3] = float("nan")
    q[0, 20, 0] *= 4096                             # a large score in the same group
    cfg = abi.window_config(1, 90, 90, 4, 2, dqk, dv, 8, 0)
    out, lse = abi.window_forward(cfg, q, k, v)
    dq, dk, dvv = abi.window_backward(cfg, q, k, v, out, lse, d_out)
    for x in (out, lse.unsqueeze(-1), dq):
        assert x[0, 50, 1].isnan().all() and x[0, 50, 0].isfinite().all() and x[0, 49, 1].isfinite().all()
    for x in (dk, dvv):
        assert x[0, 0, 43:51].isnan().any(-1).all() and x[0, 1].isfinite().all()


@pytest.mark.parametrize("dims", [(64, 64), (128, 128), (192, 128)], ids=str)
@pytest.mark.parametrize("first", [0, 60, 190, 336])
def test_dq_shows_the_part_of_every_single_key(first, dims):
    """Keys first + c, c < 64, are unit vectors e_c and all others zero, so column c of dq is scale ds of
    one key: a key too many or too few in any row changes its column by many times its bound."""
    dqk, dv = dims
    T, Hq, Hkv, W, ns = 400, 6, 2, 130, 70
    g = torch.Generator(device="cuda")
    g.manual_seed(15)
    r = lambda *s: torch.randn(*s, generator=g, device="cuda").to(torch.bfloat16)  # noqa: E731
    q, v, d_out = r(1, T, Hq, dqk), r(1, Hkv, T, dv), r(1, T, Hq, dv)
    k = torch.zeros(1, Hkv, T, dqk, dtype=torch.bfloat16, device="cuda")
    c = torch.arange(64, device="cuda")
    k[:, :, first + c, c] = 1
    cfg = abi.window_config(1, T, T, Hq, Hkv, dqk, dv, W, ns)
    out, lse = abi.window_forward(cfg, q, k, v)
    dq = abi.window_backward(cfg, q, k, v, out, lse, d_out)[0]
    vis = visible(T, T, 0, W, ns, "cuda")
    value, bound = window_ref(q, k, v, vis, cfg.scale, d_out)["dq"]
    check(dq, (value, bound), "dq")
    part = vis[:, first:first + 64]                              # [T, 64]
    ratio = (value.abs() / bound)[0, :, :, :64].transpose(1, 2)[part]
    assert float(ratio.median()) > 10
    assert not dq[0, :, :, :64].transpose(1, 2)[~part].any()
