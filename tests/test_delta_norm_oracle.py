"""Pins of the oracle's gated delta rule and layer norm (CPU, fp64): closed forms, and the
gradients against central differences."""
import numpy as np
import pytest
import torch

import oracle


def rand_delta(b=2, L=5, H=4, K=2, P=3, N=4, seed=0):
    r = np.random.default_rng(seed)
    return dict(q=r.normal(size=(b, L, K, N)), k=r.normal(size=(b, L, K, N)), v=r.normal(size=(b, L, H, P)),
                a=-r.uniform(0, 0.5, (b, L, H)), beta=r.uniform(0, 1, (b, L, H)),
                initial_state=r.normal(size=(b, H, P, N)))


def test_no_keys_gives_decayed_state():
    d = rand_delta()
    d["k"][:] = 0
    y, S = oracle.delta_rule(**d, scale=0.5)
    decay = np.exp(d["a"].cumsum(1))
    assert np.allclose(S, d["initial_state"] * decay[:, -1][..., None, None])
    qh = np.repeat(d["q"], 2, axis=2)
    assert np.allclose(y[:, 2], 0.5 * np.einsum("bhpn,bhn->bhp", d["initial_state"] * decay[:, 2][..., None, None], qh[:, 2]))


def test_unit_key_with_full_step_replaces_the_answer():
    """beta = 1 and |k| = 1: afterwards the state answers the key with the value."""
    d = rand_delta(L=1)
    d["k"] /= np.linalg.norm(d["k"], axis=-1, keepdims=True)
    d["beta"][:] = 1
    d["q"] = d["k"]
    y, _ = oracle.delta_rule(**d)
    assert np.allclose(y, d["v"])


def test_without_the_correction_it_is_the_dual():
    """Mutually orthogonal keys and a zero start: the correction vanishes, and the rule is the
    state-space dual with C = q, B = k, x = beta v."""
    r = np.random.default_rng(3)
    L, N = 4, 6
    k = np.linalg.qr(r.normal(size=(N, N)))[0][:L].reshape(1, L, 1, N)
    q, v = r.normal(size=(1, L, 1, N)), r.normal(size=(1, L, 1, 5))
    a, beta = -r.uniform(0, 0.5, (1, L, 1)), r.uniform(0, 1, (1, L, 1))
    y, S = oracle.delta_rule(q, k, v, a, beta)
    yr, Sr = oracle.ssd_loop(beta[..., None] * v, a, k, q)
    assert np.allclose(y, yr) and np.allclose(S, Sr)


def test_minus_infinity_forgets():
    d = rand_delta(L=6)
    d["a"][:, 3] = -np.inf
    y, S = oracle.delta_rule(**d)
    tail = {n: d[n][:, 3:] for n in ("q", "k", "v", "a", "beta")}
    y2, S2 = oracle.delta_rule(**tail)
    assert np.allclose(y[:, 3:], y2) and np.allclose(S, S2)


def test_delta_gradients_against_differences():
    d = rand_delta(b=1, L=4, H=2, K=1, P=2, N=3, seed=1)
    r = np.random.default_rng(2)
    dy, dS = r.normal(size=d["v"].shape), r.normal(size=d["initial_state"].shape)

    def loss(**kw):
        y, S = oracle.delta_rule(**kw, scale=0.7)
        return (dy * y).sum() + (dS * S).sum()

    g = oracle.delta_rule_bwd(dy, **d, dfinal_state=dS, scale=0.7)
    for name in d:
        got = g["d" + name]
        for i in np.ndindex(d[name].shape):
            h = 1e-6
            up, down = {n: t.copy() for n, t in d.items()}, {n: t.copy() for n, t in d.items()}
            up[name][i] += h
            down[name][i] -= h
            # central difference: error h^2 f''' and 2^-53 |f| / h, both below 1e-8 here
            assert abs((loss(**up) - loss(**down)) / (2 * h) - got[i]) < 1e-7 * max(1, abs(got[i])), (name, i)


@pytest.mark.parametrize("affine", [True, False])
def test_layer_norm_against_torch_and_differences(affine):
    r = np.random.default_rng(5)
    x, dy = r.normal(size=(3, 7)) * 2 + 1, r.normal(size=(3, 7))
    w, b = (r.normal(size=7), r.normal(size=7)) if affine else (None, None)
    y, mean, rstd = oracle.layer_norm(x, w, b, eps=1e-3)
    tx = torch.tensor(x, requires_grad=True)
    tw, tb = (torch.tensor(t, requires_grad=True) if t is not None else None for t in (w, b))
    ty = torch.nn.functional.layer_norm(tx, (7,), tw, tb, eps=1e-3)
    assert np.allclose(y, ty.detach().numpy())
    ty.backward(torch.tensor(dy))
    dx, dw, db = oracle.layer_norm_bwd(dy, x, w, mean, rstd)
    assert np.allclose(dx, tx.grad.numpy())
    if affine:
        assert np.allclose(dw, tw.grad.numpy()) and np.allclose(db, tb.grad.numpy())
    for i in np.ndindex(x.shape):
        h, up, down = 1e-6, x.copy(), x.copy()
        up[i] += h
        down[i] -= h
        diff = ((oracle.layer_norm(up, w, b, 1e-3)[0] - oracle.layer_norm(down, w, b, 1e-3)[0]) * dy).sum() / (2 * h)
        assert abs(diff - dx[i]) < 1e-7
