"""Failure detection of the window attention's tensor-core kernels, without a GPU fault: their bounded
waits run out under a short limit, the kernels report NSA_ERR_TIMEOUT and return, and later calls are
correct."""
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
