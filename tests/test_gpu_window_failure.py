"""Failure detection of the window attention's tensor-core kernels, without a GPU fault: their bounded
waits run out under a short limit, the kernels report NSA_ERR_TIMEOUT and return, and later calls are
correct; a wait's limit counts the time of its own kernel, not of the one before it in the stream."""
import pytest
import torch

from dynamic_block_sparse_scoring_b200 import abi
from tests.window_ref import check, visible, window_ref

pytestmark = pytest.mark.gpu

TIMEOUT = 5


def _inputs(g, B, Tq, Tk, Hq, Hkv, dqk, dv):
    r = lambda *s: torch.randn(*s, generator=g, device="cuda").to(torch.bfloat16)  # noqa: E731
    return dict(q=r(B, Tq, Hq, dqk), k=r(B, Hkv, Tk, dqk), v=r(B, Hkv, Tk, dv)), r(B, Tq, Hq, dv)


@pytest.mark.parametrize("dims", [(192, 128), (64, 64)], ids=str)
@pytest.mark.parametrize("planes", [2, 160])
def test_waits_run_out_and_the_next_calls_are_correct(planes, dims):
    dqk, dv = dims
    T, W, ns = 400, 130, 5
    g = torch.Generator(device="cuda")
    g.manual_seed(31)
    x, d_out = _inputs(g, 1, T, T, planes, planes, dqk, dv)
    cfg = abi.window_config(1, T, T, planes, planes, dqk, dv, W, ns)
    out, lse = abi.window_forward(cfg, **x)
    assert abi.nsa_get_device_status() == 0
    abi.nsa_set_wait_limit_ns(1)
    try:
        abi.window_forward(cfg, **x)
        forward = abi.nsa_get_device_status()
        abi.window_backward(cfg, **x, out=out, lse=lse, d_out=d_out)
        backward = abi.nsa_get_device_status()
    finally:
        abi.nsa_set_wait_limit_ns(0)
    assert forward == TIMEOUT and backward == TIMEOUT
    out, lse = abi.window_forward(cfg, **x)
    grads = abi.window_backward(cfg, **x, out=out, lse=lse, d_out=d_out)
    assert abi.nsa_get_device_status() == 0
    ref = window_ref(x["q"], x["k"], x["v"], visible(T, T, 0, W, ns, "cuda"), cfg.scale, d_out)
    for n, got in zip(("out", "lse", "dq", "dk", "dv"), (out, lse) + grads):
        check(got, ref[n], n)


def test_a_long_query_kernel_does_not_use_up_the_key_kernels_limit():
    """A few queries that see two million keys: one CTA walks them all for dq (some 30 ms), while the
    dk/dv kernel stands ready on the other SMs.  With a limit of 3 ms its waits must not run out."""
    Tq, Tk, d = 64, 2_000_000, 64
    g = torch.Generator(device="cuda")
    g.manual_seed(32)
    x, d_out = _inputs(g, 1, Tq, Tk, 1, 1, d, d)
    cfg = abi.window_config(1, Tq, Tk, 1, 1, d, d, Tk, 0, Tk - Tq)
    out, lse = abi.window_forward(cfg, **x)
    want = abi.window_backward(cfg, **x, out=out, lse=lse, d_out=d_out)
    assert abi.nsa_get_device_status() == 0
    abi.nsa_set_wait_limit_ns(3_000_000)
    try:
        got = abi.window_backward(cfg, **x, out=out, lse=lse, d_out=d_out)
        status = abi.nsa_get_device_status()
    finally:
        abi.nsa_set_wait_limit_ns(0)
    assert status == 0
    for a, b in zip(got, want):
        assert torch.equal(a, b)
    assert want[1].any() and want[2].any()
