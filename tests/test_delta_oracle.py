"""The fp64 references of the gated delta rule and layer norm against closed forms,
the SSD oracle and differences (CPU)."""
import numpy as np
import pytest

import oracle
from oracle import delta


def draw(rng, b=2, T=7, H=4, P=3, N=5, G=2):
    unit = lambda x: x / np.linalg.norm(x, axis=-1, keepdims=True)
    return dict(q=unit(rng.standard_normal((b, T, G, N))), k=unit(rng.standard_normal((b, T, G, N))),
                v=rng.standard_normal((b, T, H, P)), g=-rng.uniform(0, 1, (b, T, H)), beta=rng.uniform(0, 1, (b, T, H)))


def test_orthonormal_keys_reduce_to_the_plain_recurrence():
    """With keys that are orthogonal to each other nothing is erased: S_t = sum of
    decayed beta v k^T, so y is a masked sum."""
    rng = np.random.default_rng(0)
    T, N, P = 5, 5, 3
    k = np.eye(N)[None, :, None]
    x = dict(q=rng.standard_normal((1, T, 1, N)), k=k, v=rng.standard_normal((1, T, 1, P)),
             g=-rng.uniform(0, 1, (1, T, 1)), beta=rng.uniform(0, 1, (1, T, 1)))
    y, S = delta.gdr_forward(**x, scale=0.5)
    cs = np.cumsum(x["g"][0, :, 0])
    want = np.zeros((T, P))
    for t in range(T):
        for s in range(t + 1):
            want[t] += 0.5 * np.exp(cs[t] - cs[s]) * x["beta"][0, s, 0] * x["v"][0, s, 0] * x["q"][0, t, 0, s]
    np.testing.assert_allclose(y[0, :, 0], want, rtol=1e-12, atol=1e-14)


def test_a_key_written_twice_holds_the_last_value():
    """beta = 1 and one unit key, no decay: the state returns the newest value."""
    rng = np.random.default_rng(1)
    k = np.zeros((1, 4, 1, 6))
    k[..., 2] = 1
    v = rng.standard_normal((1, 4, 1, 3))
    y, S = delta.gdr_forward(k, k, v, np.zeros((1, 4, 1)), np.ones((1, 4, 1)))
    np.testing.assert_allclose(y, v, rtol=1e-13)


def test_without_erasing_it_is_the_ssd():
    """The rule with u = v (the erased part added back) is the SSD recurrence: feed
    v' = v + e^g S k from the SSD's own states."""
    rng = np.random.default_rng(2)
    x = draw(rng, b=1, G=2)
    A = -np.ones(4)
    ref = oracle.forward(x["v"], -x["g"] * 1.0, A, x["k"], x["q"], dt_softplus=False)
    # SSD: h = e^{dt A} h + dt x B^T with dt = -g, A = -1: beta = dt, v as is
    S = np.zeros((1, 4, 3, 5))
    v2 = np.zeros_like(x["v"])
    for t in range(7):
        kt = np.repeat(x["k"][:, t], 2, axis=1)
        v2[:, t] = x["v"][:, t] + (S * np.exp(x["g"][:, t])[..., None, None] * kt[:, :, None]).sum(-1)
        _, S = delta.gdr_step(x["q"][:, t], x["k"][:, t], v2[:, t], x["g"][:, t], -x["g"][:, t], S)
    y, fin = delta.gdr_forward(x["q"], x["k"], v2, x["g"], -x["g"])
    np.testing.assert_allclose(y, ref.y, rtol=1e-10, atol=1e-12)
    np.testing.assert_allclose(fin, ref.final_states, rtol=1e-10, atol=1e-12)


@pytest.mark.parametrize("packed", [False, True])
def test_backward_against_differences(packed):
    rng = np.random.default_rng(3)
    x = draw(rng, b=1 if packed else 2, T=9)
    n = 4 if packed else 2
    kw = dict(seq_idx=np.array([0, 0, 0, 1, 1, 3, 3, 3, 3], np.int32), nseq=4) if packed else {}
    init, dfin = rng.standard_normal((n, 4, 3, 5)), rng.standard_normal((n, 4, 3, 5))
    dy = rng.standard_normal(x["v"].shape)

    def loss(x, init):
        y, f = delta.gdr_forward(**x, scale=0.7, initial_states=init, **kw)
        return (y * dy).sum() + (f * dfin).sum()

    got = delta.gdr_backward(**x, dy=dy, scale=0.7, initial_states=init, dfinal_states=dfin, **kw)
    h = 1e-6
    for name in ("q", "k", "v", "g", "beta", "initial_states"):
        d = rng.standard_normal((init if name == "initial_states" else x[name]).shape)
        if name == "initial_states":
            num = (loss(x, init + h * d) - loss(x, init - h * d)) / (2 * h)
        else:
            num = (loss(dict(x, **{name: x[name] + h * d}), init) - loss(dict(x, **{name: x[name] - h * d}), init)) / (2 * h)
        # differences in 64 bits: truncation h^2 and rounding 1e-16 / h, both about 1e-10 of the loss's size
        np.testing.assert_allclose((got["d" + name] * d).sum(), num, rtol=1e-6, atol=1e-7)


def test_layer_norm_backward_against_differences():
    rng = np.random.default_rng(4)
    x, dy = rng.standard_normal((5, 9)), rng.standard_normal((5, 9))
    w, b = rng.standard_normal(9), rng.standard_normal(9)
    f = lambda x, w, b: (delta.layer_norm(x, w, b)[0] * dy).sum()
    _, mean, rstd = delta.layer_norm(x, w, b)
    dx, dw, db = delta.layer_norm_backward(x, dy, mean, rstd, w)
    h = 1e-6
    for i, (a, da) in enumerate(((x, dx), (w, dw), (b, db))):
        d = rng.standard_normal(a.shape)
        args = [x, w, b]
        up, dn = list(args), list(args)
        up[i], dn[i] = a + h * d, a - h * d
        np.testing.assert_allclose((da * d).sum(), (f(*up) - f(*dn)) / (2 * h), rtol=1e-6, atol=1e-7)
