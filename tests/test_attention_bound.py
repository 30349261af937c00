"""The attention's bound (attention_bound) is tight enough: outputs whose softmax weights are held in too few bits are
outside it, those of the weights as the kernel holds them inside (CPU)."""
import numpy as np
import pytest

import attention_bound as ab


def outside(q, k, v, scale, t, ct, part, parts, up):
    o, tol, _, _ = ab.bound(q, k, v, scale, t, ct)
    return (np.abs(ab.with_weights_as(q, k, v, scale, t, part, parts, up) - o) > tol).sum()


@pytest.mark.parametrize("t,ct,part", [("f16", "f16", "f16"), ("bf16", "bf16", "bf16"), ("f16", "e4m3", "f16")])
@pytest.mark.parametrize("n", [3, 17, 40])
def test_one_part_a_weight_is_seen(t, ct, part, n):
    g = np.random.default_rng(n)
    one = two = 0
    for _ in range(20):
        q, k, v = (ab.rounded(g.standard_normal(s), t) for s in ((64,), (n, 64), (n, 64)))
        one += outside(q, k, v, 0.125, t, ct, part, 1, 15 if part == "f16" else 0)
        two += outside(q, k, v, 0.125, t, ct, part, 2, 15 if part == "f16" else 0)
    assert one > 20 and two == 0


@pytest.mark.parametrize("t,ct", [("f16", "f16"), ("f16", "e4m3"), ("bf16", "e4m3")])
@pytest.mark.parametrize("n,above", [(1000, 14.0), (1000, 17.0), (20000, 16.0), (300, 22.0)])
def test_small_weights_that_are_lost_are_seen(t, ct, n, above):
    g = np.random.default_rng(n)
    q = ab.rounded(g.standard_normal((4, 64)), t)
    k, v = (ab.rounded(x, t) for x in ab.sink(g, n, 64, above, q, 0.125))
    v = v * 64
    lost = sum(outside(x, k, v, 0.125, t, ct, "f16", 2, 0) for x in q)
    held = sum(outside(x, k, v, 0.125, t, ct, "f16", 2, 15) for x in q)
    assert lost > 0 and held == 0
