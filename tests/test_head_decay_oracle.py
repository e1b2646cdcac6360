"""The fp64 reference of the per-head-decay family: against its closed form, its
gradients against central differences, the selection against a plain sort."""
import numpy as np
import pytest

from oracle import head_decay as ref


def _case(seed, T, H, Hk, Dk, Dv):
    r = np.random.default_rng(seed)
    return dict(q=r.normal(size=(T, H, Dk)), k=r.normal(size=(T, Hk, Dk)), v=r.normal(size=(T, Hk, Dv)),
                g=-r.uniform(0.0, 1.0, size=H), s0=r.normal(size=(H, Dk, Dv)))


def test_forward_closed_form():
    x = _case(1, 9, 4, 2, 3, 5)
    o, S = ref.forward(**x, scale=0.5)
    for h in range(4):
        lam = np.exp(x["g"][h])
        for t in range(9):
            want = lam ** (t + 1) * x["s0"][h].T @ x["q"][t, h]
            for j in range(t + 1):
                want = want + lam ** (t - j) * (x["q"][t, h] @ x["k"][j, h // 2]) * x["v"][j, h // 2]
            assert np.allclose(o[t, h], 0.5 * want, rtol=1e-12, atol=1e-12)


@pytest.mark.parametrize("T", [0, 1, 6])
def test_gradients_are_differences(T):
    x = _case(2, T, 4, 2, 3, 2)
    r = np.random.default_rng(3)
    d_o, ds = r.normal(size=(T, 4, 2)), r.normal(size=(4, 3, 2))

    def loss(y):
        o, S = ref.forward(**y, scale=0.7)
        return (o * d_o).sum() + (S[-1] * ds).sum()

    grads = ref.backward(**x, d_o=d_o, ds_final=ds, scale=0.7)
    eps = 1e-5
    for name, got in (("q", "dq"), ("k", "dk"), ("v", "dv"), ("g", "dg"), ("s0", "ds0")):
        for _ in range(6 if x[name].size else 0):
            at = tuple(r.integers(0, n) for n in x[name].shape)
            hi, lo = {k: v.copy() for k, v in x.items()}, {k: v.copy() for k, v in x.items()}
            hi[name][at] += eps
            lo[name][at] -= eps
            # the loss is smooth: a central difference is off by eps^2 / 6 of its third derivative, and by
            # 2^-52 |loss| / eps of rounding, both far below 1e-6 at these sizes
            assert abs((loss(hi) - loss(lo)) / (2 * eps) - grads[got][at]) < 1e-6, name


def test_selection_order_and_rules():
    nan, inf = np.nan, np.inf
    logits = np.array([[0.0, 1.0, 1.0], [nan, 0.0, 0.0], [-inf, -inf, -inf], [5.0, 5.0, 5.0]])
    # beam 0: tokens 1 and 2 tie; beam 1 and 2 offer nothing finite; beam 3 is done
    s, t, p, d = ref.select(logits, np.array([0.0, 0.0, 0.0, -1.0]), done=[0, 0, 0, 1], eos=2, pad=1)
    assert list(p) == [0, 0, 3, 0] and list(t) == [1, 2, 1, 0] and list(d) == [False, True, True, False]
    s, t, p, d = ref.select(logits[1:3], np.array([0.0, 0.0]))
    assert list(p) == [0, 0] and list(t) == [0, 1] and np.all(s == -inf)
