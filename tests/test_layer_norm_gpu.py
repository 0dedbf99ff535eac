"""GPU parity of the layer norm and its backward with the fp64 oracle.

Bounds, derived before the first run: sums of n fp32 values in a tree of lanes with short
serial runs are off by at most (n / lanes + log2 lanes + ..) 2^-24, taken as 2^-19 of the
summands' size for every width here; a mean off by d moves y by d rstd |w|, and subtracting it
from values of size X costs 2^-24 X.  With X = max|x| of the row: |err y| <= 2^-18 (1 + X rstd)
|w|max + 2^-22 |y|, plus half a step of the output type.  dx likewise, relative to rstd |g|max;
dweight and dbias: 2^-18 of the sum of magnitudes, and through xhat's error.
"""
import numpy as np
import pytest
import torch

import oracle
import selective_state_space_45_b200 as ssm
from tests.helpers import to64

pytestmark = pytest.mark.gpu
DEV = "cuda"
F32, BF16 = torch.float32, torch.bfloat16
STEP = {F32: 2.0 ** -24, BF16: 2.0 ** -8}
DIMS = [1, 2, 7, 8, 40, 64, 65, 128, 130, 256, 300, 512, 520, 768, 777, 1000, 1024, 1032, 2560, 4097, 8184, 8192]


def make(rows, dim, dtype, seed=0, offset=0.0):
    g = torch.Generator().manual_seed(seed)
    x = (torch.randn(rows, dim, generator=g) * 1.5 + offset).to(dtype).to(DEV)
    w, b = 1 + 0.3 * torch.randn(dim, generator=g), 0.3 * torch.randn(dim, generator=g)
    return x, w.to(DEV), b.to(DEV), torch.randn(rows, dim, generator=g)


def check_fwd(x, w, b, out=None, eps=1e-5):
    y, mean, rstd = ssm.layer_norm(x, w, b, eps=eps, out_dtype=out, return_stats=True)
    yr, mr, rr = oracle.layer_norm(x, w, b, eps)
    big = np.abs(to64(x)).max(-1)
    wm = 1.0 if w is None else np.abs(to64(w)).max()
    err = np.abs(to64(y) - yr)
    bound = (2.0 ** -18 * (1 + big * rr) * wm)[:, None] + (2.0 ** -22 + STEP[y.dtype]) * np.abs(yr)
    assert (err <= bound).all(), (float((err - bound).max()), x.shape)
    assert (np.abs(to64(mean) - mr) <= 2.0 ** -19 * big + 1e-30).all()
    assert (np.abs(to64(rstd) - rr) <= (2.0 ** -18 + 2.0 ** -36 * (big * rr) ** 2) * rr).all()
    return mean, rstd


def check_bwd(x, w, dy, mean, rstd):
    g = ssm.layer_norm_bwd(dy, x, w, mean, rstd)
    dxr, dwr, dbr = oracle.layer_norm_bwd(dy, x, w, mean, rstd)
    xs, r, m = to64(x), to64(rstd)[:, None], to64(mean)[:, None]
    h, d = np.abs((xs - m) * r), np.abs(to64(dy))
    hx = 2.0 ** -22 * (h + np.abs(xs) * r)                       # error of xhat itself
    gm = (d * (1 if w is None else np.abs(to64(w)))).max(-1, keepdims=True)
    hm = h.max(-1, keepdims=True)
    bound = r * gm * (2.0 ** -18 * (1 + hm) * (1 + h) + hx.max(-1, keepdims=True) * (1 + hm)) + STEP[dy.dtype] * np.abs(dxr)
    err = np.abs(to64(g["dx"]) - dxr)
    assert g["dx"].dtype == dy.dtype and (err <= bound + 1e-30).all(), (float((err / (bound + 1e-30)).max()), x.shape)
    assert (np.abs(to64(g["dweight"]) - dwr) <= 2.0 ** -18 * (d * h).sum(0) + (d * hx).sum(0) + 1e-30).all()
    assert (np.abs(to64(g["dbias"]) - dbr) <= 2.0 ** -18 * d.sum(0) + 1e-30).all()
    return g


@pytest.mark.parametrize("dim", DIMS)
@pytest.mark.parametrize("dtype,other", [(F32, F32), (BF16, BF16), (F32, BF16), (BF16, F32)])
def test_rows(cuda_lib, dim, dtype, other):
    for rows in (1, 3, 37):
        x, w, b, dy = make(rows, dim, dtype, seed=dim + rows)
        mean, rstd = check_fwd(x, w, b, other)
        check_bwd(x, w, dy.to(other).to(DEV), mean, rstd)


@pytest.mark.parametrize("rows,dim", [(5000, 64), (20001, 32), (3001, 768), (1500, 2560), (700, 8192), (1, 8192)])
def test_many_rows(cuda_lib, rows, dim):
    """More rows than the grid holds at once: every group walks several."""
    x, w, b, dy = make(rows, dim, BF16, seed=rows)
    mean, rstd = check_fwd(x, w, b)
    check_bwd(x, w, dy.to(BF16).to(DEV), mean, rstd)


@pytest.mark.parametrize("rows,dim,dtype", [(160001, 64, BF16), (310003, 40, BF16), (170005, 32, F32), (80001, 128, BF16),
                                            (60007, 120, F32), (40011, 200, BF16)])
def test_more_rows_than_steps_of_the_whole_grid(cuda_lib, rows, dim, dtype):
    """Enough narrow rows that a group takes several a step, the last step partly past the end."""
    x, w, b, _ = make(rows, dim, dtype, seed=rows)
    check_fwd(x, w, b)


@pytest.mark.parametrize("dim", [64, 100, 1024, 3000])
def test_without_weight_or_bias(cuda_lib, dim):
    x, w, b, dy = make(9, dim, F32, seed=dim)
    mean, rstd = check_fwd(x, None, None)
    check_fwd(x, w, None)
    check_fwd(x, None, b)
    check_bwd(x, None, dy.to(DEV), mean, rstd)
    dx = torch.empty_like(x)
    ssm.ssm_layer_norm_bwd(dy.to(DEV), x, w, mean, rstd, dx)                 # no parameter gradients asked for
    assert torch.equal(dx, ssm.layer_norm_bwd(dy.to(DEV), x, w, mean, rstd)["dx"])


def test_hard_rows(cuda_lib):
    """Constant rows (variance 0), rows far from zero, tiny and huge rows."""
    x, w, b, dy = make(6, 512, F32, seed=3)
    x[0] = 3.25
    x[1] = 0
    x[2] += 4096
    x[3] *= 1e-18
    x[4] *= 1e15
    mean, rstd = check_fwd(x, w, b)
    check_bwd(x[[2, 3, 5]].contiguous(), w, dy[[2, 3, 5]].to(DEV), mean[[2, 3, 5]].contiguous(), rstd[[2, 3, 5]].contiguous())
    y = ssm.layer_norm(x, w, b)
    assert torch.equal(y[1], b)


def test_a_bad_row_stays_alone(cuda_lib):
    """NaN and inf in one row leave the other rows' outputs as they were."""
    for dim in (64, 768, 2560):
        x, w, b, _ = make(40, dim, BF16, seed=dim)
        y = ssm.layer_norm(x, w, b)
        z = x.clone()
        z[7, 3], z[20, dim - 1] = float("nan"), float("inf")
        yz = ssm.layer_norm(z, w, b)
        keep = [i for i in range(40) if i not in (7, 20)]
        assert torch.equal(y[keep], yz[keep]) and bool(yz[7].isnan().all()) and bool(yz[20].isnan().all())


def test_leading_dimensions_and_guards(cuda_lib):
    x, w, b, dy = make(2 * 3 * 5, 72, BF16, seed=1)
    y = ssm.layer_norm(x.reshape(2, 3, 5, 72), w, b)
    assert y.shape == (2, 3, 5, 72) and torch.equal(y.reshape(30, 72), ssm.layer_norm(x, w, b))
    out = torch.full((30 * 72 + 64,), 7.0, device=DEV, dtype=BF16)
    ssm.ssm_layer_norm_fwd(x, w, b, out[:30 * 72].reshape(30, 72))
    assert torch.equal(out[:30 * 72].reshape(30, 72), y.reshape(30, 72)) and bool((out[30 * 72:] == 7).all())


def test_no_rows(cuda_lib):
    x = torch.empty(0, 64, device=DEV)
    w = torch.ones(64, device=DEV)
    y, mean, rstd = ssm.layer_norm(x, w, None, return_stats=True)
    g = ssm.layer_norm_bwd(x, x, w, mean, rstd)
    assert y.shape == (0, 64) and not g["dweight"].any() and not g["dbias"].any()


def test_results_do_not_vary_and_replay(cuda_lib):
    x, w, b, dy = make(3000, 776, BF16, seed=5)
    dy = dy.to(BF16).to(DEV)
    y, mean, rstd = ssm.layer_norm(x, w, b, return_stats=True)
    g = ssm.layer_norm_bwd(dy, x, w, mean, rstd)
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        yc, mc, rc = ssm.layer_norm(x, w, b, return_stats=True)
        gc = ssm.layer_norm_bwd(dy, x, w, mc, rc)
    for _ in range(2):
        graph.replay()
        assert torch.equal(yc, y) and all(torch.equal(gc[n], g[n]) for n in g)
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        g2 = ssm.layer_norm_bwd(dy, x, w, mean, rstd)
    s.synchronize()
    assert all(torch.equal(g2[n], g[n]) for n in g)


# ---- the operators together ----------------------------------------------------------------


def test_block_forward_and_gradients(cuda_lib):
    """A residual block as it would be used: norm, projections to unit queries and keys, the
    delta rule, a norm per head, the output projection -- and its whole gradient, against
    autograd in fp64 over the token-by-token definition.  fp32 throughout: the operators'
    bounds are 2^-15 and below, the chain of six products in fp32 adds as much again: 2^-13."""
    torch.backends.cuda.matmul.allow_tf32 = False
    B, L, D, H, K, P, N = 2, 70, 96, 4, 2, 32, 32
    g = torch.Generator().manual_seed(0)
    shapes = dict(x=(B, L, D), w1=(D,), b1=(D,), wq=(D, K * N), wk=(D, K * N), wv=(D, H * P), wa=(D, H), wb=(D, H), w2=(P,),
                  b2=(P,), wo=(H * P, D))
    prm = {n: (torch.randn(s, generator=g) * (0.15 if n.startswith("w") and len(s) == 2 else 1) + (n in ("w1", "w2"))).to(DEV)
           for n, s in shapes.items()}
    up = torch.randn(B, L, D, generator=g).to(DEV)
    scale = N ** -0.5

    def unit(t):
        return t / t.norm(dim=-1, keepdim=True)

    def reference(p):
        h = torch.nn.functional.layer_norm(p["x"], (D,), p["w1"], p["b1"])
        q, k = (unit((h @ p[n]).reshape(B, L, K, N)).repeat_interleave(H // K, 2) for n in ("wq", "wk"))
        v = (h @ p["wv"]).reshape(B, L, H, P)
        a, beta = -torch.nn.functional.softplus(h @ p["wa"]), torch.sigmoid(h @ p["wb"])
        S, ys = torch.zeros(B, H, P, N, device=DEV, dtype=torch.float64), []
        for t in range(L):
            S = S * a[:, t].exp()[..., None, None]
            e = v[:, t] - (S @ k[:, t][..., None])[..., 0]
            S = S + (beta[:, t][..., None] * e)[..., None] * k[:, t][..., None, :]
            ys.append(scale * (S @ q[:, t][..., None])[..., 0])
        o = torch.nn.functional.layer_norm(torch.stack(ys, 1), (P,), p["w2"], p["b2"])
        return p["x"] + o.reshape(B, L, H * P) @ p["wo"]

    class Norm(torch.autograd.Function):
        @staticmethod
        def forward(ctx, x, w, b):
            y, mean, rstd = ssm.layer_norm(x, w, b, return_stats=True)
            ctx.save_for_backward(x, w, mean, rstd)
            return y

        @staticmethod
        def backward(ctx, dy):
            d = ssm.layer_norm_bwd(dy.contiguous(), *ctx.saved_tensors)
            return d["dx"], d["dweight"], d["dbias"]

    class Delta(torch.autograd.Function):
        @staticmethod
        def forward(ctx, *t):
            ctx.save_for_backward(*t)
            return ssm.delta_rule(*t, scale=scale, return_final_state=False)

        @staticmethod
        def backward(ctx, dy):
            d = ssm.delta_rule_bwd(dy.contiguous(), *ctx.saved_tensors, scale=scale)
            return d["dq"], d["dk"], d["dv"], d["da"], d["dbeta"]

    def block(p):
        h = Norm.apply(p["x"], p["w1"], p["b1"])
        q, k = (unit((h @ p[n]).reshape(B, L, K, N)).contiguous() for n in ("wq", "wk"))
        v = (h @ p["wv"]).reshape(B, L, H, P)
        a, beta = -torch.nn.functional.softplus(h @ p["wa"]), torch.sigmoid(h @ p["wb"])
        o = Norm.apply(Delta.apply(q, k, v, a, beta), p["w2"], p["b2"])
        return p["x"] + o.reshape(B, L, H * P) @ p["wo"]

    ours = {n: t.clone().requires_grad_() for n, t in prm.items()}
    ref = {n: t.double().requires_grad_() for n, t in prm.items()}
    yo, yr = block(ours), reference(ref)
    assert float(((yo.double() - yr).norm() / yr.norm()).detach()) <= 2.0 ** -13
    yo.backward(up)
    yr.backward(up.double())
    for n in prm:
        err = float((ours[n].grad.double() - ref[n].grad).norm() / ref[n].grad.norm())
        assert err <= 2.0 ** -12, (n, err)
