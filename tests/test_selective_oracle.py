"""Pins of the fp64 oracle of the selective scan, the convolution, RMS norm and the 8-bit product: closed forms,
and every gradient against central differences (CPU)."""
import numpy as np
import pytest
import torch

from oracle import selective as sel


def rnd(rng, *shape):
    return rng.standard_normal(shape)


def scan_case(rng, packed, gate=True):
    dim, N, G = 6, 3, 2
    lengths = [4, 1, 0, 3] if packed else None
    b, T = (1, 8) if packed else (2, 5)
    rows = len(lengths) if packed else b
    a = dict(x=rnd(rng, b, T, dim), dt=rnd(rng, b, T, dim), A=-np.exp(rnd(rng, dim, N)), B=rnd(rng, b, T, G, N), C=rnd(rng, b, T, G, N),
             D=rnd(rng, dim), z=rnd(rng, b, T, dim) if gate else None, dt_bias=rnd(rng, dim), init=rnd(rng, rows, dim, N))
    return a, lengths, rnd(rng, b, T, dim), rnd(rng, rows, dim, N)


@pytest.mark.parametrize("packed", [False, True])
@pytest.mark.parametrize("softplus", [False, True])
def test_scan_gradients_against_differences(packed, softplus):
    rng = np.random.default_rng(0)
    a, lengths, dy, df = scan_case(rng, packed)

    def loss(**kw):
        y, f = sel.scan_forward(**{**a, **kw}, softplus=softplus, lengths=lengths)
        return (y * dy).sum() + (f * df).sum()

    g = sel.scan_backward(**a, dy=dy, dfinal=df, softplus=softplus, lengths=lengths)
    # without softplus a step may be negative and the state grow: each loss is a sum of terms of size S, off by
    # some 8 roundings of 2^-53 S, which the difference divides by 1e-5: 9e-11 S
    y, f = sel.scan_forward(**a, softplus=softplus, lengths=lengths)
    S = np.abs(y * dy).sum() + np.abs(f * df).sum()
    names = {"x": "dx", "dt": "ddt", "A": "dA", "B": "dB", "C": "dC", "D": "dD", "z": "dz", "dt_bias": "ddt_bias", "init": "dinitial_states"}
    for n, dn in names.items():
        for _ in range(6):
            at = tuple(rng.integers(0, s) for s in a[n].shape)
            e = np.zeros_like(a[n])
            e[at] = 1e-5
            num = (loss(**{n: a[n] + e}) - loss(**{n: a[n] - e})) / 2e-5
            assert abs(num - g[dn][at]) <= 1e-7 * max(1, abs(num)) + 9e-11 * S, (n, at)


def test_scan_closed_form():
    """One channel, one state, constant inputs: a geometric sum."""
    T, dt, A, x, B, C = 7, 0.3, -0.8, 1.5, 0.7, -1.2
    one = lambda v: np.full((1, T, 1), v)
    y, f = sel.scan_forward(one(x), one(dt), np.array([[A]]), one(B)[..., None], one(C)[..., None], softplus=False)
    a = np.exp(dt * A)
    h = dt * x * B * (1 - a ** np.arange(1, T + 1)) / (1 - a)
    assert np.allclose(y[0, :, 0], C * h, rtol=1e-13) and np.allclose(f, h[-1])


def test_scan_with_one_rate_a_head_is_the_ssd():
    """Channels of a head with one rate and step: the recurrence of the SSD oracle."""
    import oracle
    rng = np.random.default_rng(1)
    b, T, H, P, N = 1, 9, 2, 16, 16
    t = lambda a: torch.from_numpy(np.ascontiguousarray(a, dtype=np.float32))
    x, dt, A, B, C, D = t(rnd(rng, b, T, H, P)), t(rnd(rng, b, T, H)), t(-np.exp(rnd(rng, H))), t(rnd(rng, b, T, 1, N)), t(rnd(rng, b, T, 1, N)), t(rnd(rng, H))
    ref = oracle.forward(x, dt, A, B, C, D, None)
    y, f = sel.scan_forward(x.reshape(b, T, H * P), dt.repeat_interleave(P, 2), A.repeat_interleave(P)[:, None].expand(H * P, N), B, C,
                            D.repeat_interleave(P))
    assert np.allclose(y.reshape(b, T, H, P), ref.y, rtol=1e-9, atol=1e-12)
    assert np.allclose(f.reshape(b, H, P, N), ref.final_states, rtol=1e-9, atol=1e-12)


@pytest.mark.parametrize("K", [1, 2, 4])
@pytest.mark.parametrize("silu", [False, True])
@pytest.mark.parametrize("packed", [False, True])
def test_conv_gradients_against_differences(K, silu, packed):
    rng = np.random.default_rng(2)
    dim, lengths = 3, [5, 1, 0, 2] if packed else None
    b, T = (1, 8) if packed else (2, 4)
    rows = 4 if packed else b
    a = dict(x=rnd(rng, b, T, dim), weight=rnd(rng, dim, K), bias=rnd(rng, dim), window=rnd(rng, rows, K - 1, dim))
    dy, df = rnd(rng, b, T, dim), rnd(rng, rows, K - 1, dim)

    def loss(**kw):
        y, f = sel.conv_forward(**{**a, **kw}, silu=silu, lengths=lengths)
        return (y * dy).sum() + (f * df).sum()

    g = sel.conv_backward(**a, dy=dy, dwindow=df, silu=silu, lengths=lengths)
    for n, dn in {"x": "dx", "weight": "dweight", "bias": "dbias", "window": "dinitial_window"}.items():
        for at in np.ndindex(a[n].shape):
            e = np.zeros_like(a[n])
            e[at] = 1e-5
            num = (loss(**{n: a[n] + e}) - loss(**{n: a[n] - e})) / 2e-5
            assert abs(num - g[dn][at]) <= 1e-7 * max(1, abs(num)), (n, at)


def test_conv_against_the_prologue_s_oracle():
    import oracle
    rng = np.random.default_rng(3)
    x, w, b = (torch.from_numpy(rnd(rng, *s).astype(np.float32)) for s in ((2, 11, 48), (48, 4), (48,)))
    rx, rB, rC = oracle.conv1d_silu(x, w, 1, 16, 1, 16, b)
    y, f = sel.conv_forward(x, w, b)
    assert np.allclose(y, np.concatenate([a.reshape(2, 11, 16) for a in (rx, rB, rC)], -1), rtol=1e-12, atol=1e-12)
    assert np.array_equal(f, x[:, -3:].double().numpy())


def test_rms_gradients_against_differences():
    rng = np.random.default_rng(4)
    r, w, dy, dr = rnd(rng, 3, 7), rnd(rng, 7), rnd(rng, 3, 7), rnd(rng, 3, 7)
    loss = lambda r, w: (sel.rms_norm(r, w)[0] * dy).sum() + (r * dr).sum()
    g, dw, _ = sel.rms_norm_backward(r, dy, sel.rms_norm(r, w)[1], w, dr)
    for at in np.ndindex(r.shape):
        e = np.zeros_like(r)
        e[at] = 1e-5
        assert abs((loss(r + e, w) - loss(r - e, w)) / 2e-5 - g[at]) <= 1e-7
    for i in range(7):
        e = np.zeros(7)
        e[i] = 1e-5
        assert abs((loss(r, w + e) - loss(r, w - e)) / 2e-5 - dw[i]) <= 1e-7


def test_8bit_and_product():
    rng = np.random.default_rng(5)
    y = rnd(rng, 3, 300)
    y[1, :128] = 0
    s, q = sel.to_8bit(y)
    assert s.shape == (3, 3) and s[1, 0] == 2.0 ** -126 and np.allclose(np.abs(q[0, :128]).max(), 448)
    assert np.allclose(q * np.repeat(s, 128, -1)[:, :300], y)
    f8 = lambda a: torch.from_numpy(a.astype(np.float32)).to(torch.float8_e4m3fn)
    w = rnd(rng, 130, 300)
    sw = np.abs(rnd(rng, 2, 3))
    out, size = sel.matmul_fp8(f8(q), s, f8(w), sw, np.ones(130))
    i, j = 2, 129
    want = sum(sel.f64(f8(q))[i, k] * s[i, k // 128] * sel.f64(f8(w))[j, k] * sw[1, k // 128] for k in range(300)) + 1
    assert abs(out[i, j] - want) <= 1e-12 * size[i, j]
