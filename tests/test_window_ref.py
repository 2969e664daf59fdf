"""The 64-bit window attention that the GPU tests compare with, against differences and hand values."""
import math

import torch

from tests.window_ref import visible, window_ref


def _case(T=9, Tk=11, q0=2, Hq=4, Hkv=2, d=5, dv=3, window=4, sink=2, B=2):
    g = torch.Generator().manual_seed(3)
    r = lambda *s: torch.randn(*s, generator=g, dtype=torch.float64)  # noqa: E731
    return (r(B, T, Hq, d), r(B, Hkv, Tk, d), r(B, Hkv, Tk, dv), visible(T, Tk, q0, window, sink, "cpu"),
            0.7, r(B, T, Hq, dv))


def test_gradients_are_those_of_differences():
    q, k, v, vis, scale, do = _case()
    ref = window_ref(q, k, v, vis, scale, do)
    loss = lambda q, k, v: float((window_ref(q, k, v, vis, scale)["out"][0] * do).sum())  # noqa: E731
    h = 1e-5
    for name, x, args in [("dq", q, lambda y: (y, k, v)), ("dk", k, lambda y: (q, y, v)),
                          ("dv", v, lambda y: (q, k, y))]:
        grad = ref[name][0].reshape(-1)
        for i in range(0, x.numel(), 7):
            up, down = x.clone().reshape(-1), x.clone().reshape(-1)
            up[i] += h
            down[i] -= h
            fd = (loss(*args(up.view_as(x))) - loss(*args(down.view_as(x)))) / (2 * h)
            assert abs(fd - float(grad[i])) <= 1e-8 + 1e-6 * abs(fd), (name, i)


def test_visibility_by_hand():
    vis = visible(4, 6, 2, 2, 1, "cpu")          # positions 2..5, window 2, one sink
    assert vis.int().tolist() == [[1, 1, 1, 0, 0, 0], [1, 0, 1, 1, 0, 0], [1, 0, 0, 1, 1, 0],
                                  [1, 0, 0, 0, 1, 1]]


def test_uniform_scores_average_the_visible_values():
    q = torch.zeros(1, 3, 1, 4)
    k = torch.ones(1, 1, 3, 4)
    v = torch.tensor([[[[1.0], [3.0], [8.0]]]])
    ref = window_ref(q, k, v, visible(3, 3, 0, 2, 0, "cpu"), 1.0)
    assert torch.allclose(ref["out"][0].flatten(), torch.tensor([1.0, 2.0, 5.5], dtype=torch.float64))
    assert torch.allclose(ref["lse"][0].flatten(),
                          torch.tensor([0.0, math.log(2), math.log(2)], dtype=torch.float64))


def test_a_row_without_keys_is_zero():
    q, k, v, vis, scale, _ = _case()
    vis[3] = False
    ref = window_ref(q, k, v, vis, scale)
    assert not ref["out"][0][:, 3].any() and torch.isinf(ref["lse"][0][:, 3]).all()
