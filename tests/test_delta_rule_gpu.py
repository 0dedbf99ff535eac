"""GPU parity of the gated delta rule (forward, decode tokens, backward) with the fp64 oracle.

Bounds, derived before the first run (per output tensor, M = max|ref|, u(t) = half a step):
  * fp32 outputs that follow the state (final state, fp32 y, da, dbeta, start-state and fp32
    gradients): every product takes operands in two fp16 pieces, off by at most 2^-22 of an
    element, and sums up to 128 terms in fp32 accumulators that cut off (2^-23 a step).  Cut
    off sums of n terms are off by at most n 2^-23 of their size, sqrt(n)-like for mixed
    signs; with the chunk's three chained products (R, T R, update) 3 * 128 * 2^-23 = 2^-14.4
    at worst.  Relative L2 error <= 2^-15 and |err| <= 2^-13 M.
  * a bf16 y: u = 2^-8 of the value, and behind it one fp16 piece per operand (2^-12 each, two
    operands): |err| <= 2^-8 |ref| + 2^-10 M.  bf16 dq, dk chain two such products (four
    roundings): 2^-8 |ref| + 2^-9 M.  bf16 dv is an fp32 value rounded: 2^-8 |ref| + 2^-13 M.
    (The kernels have taken two pieces there, too, since; the tests of rounded values hold them to it.)
  * decode tokens are fp32 arithmetic throughout: sums of 128 terms, 128 * 2^-24 = 2^-17 at
    worst per token: |err| <= 2^-16 M (+ u |ref|).
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
INF, NAN = float("inf"), float("nan")


def make(b, L, H, K, P, N, dtype=BF16, seed=0, state=True, decay=0.3):
    g = torch.Generator().manual_seed(seed)
    q, k = (torch.randn(b, L, K, N, generator=g) for _ in range(2))
    d = dict(q=(q / q.norm(dim=-1, keepdim=True)).to(dtype), k=(k / k.norm(dim=-1, keepdim=True)).to(dtype),
             v=torch.randn(b, L, H, P, generator=g).to(dtype), a=-decay * torch.rand(b, L, H, generator=g),
             beta=torch.rand(b, L, H, generator=g))
    d["initial_state"] = 0.5 * torch.randn(b, H, P, N, generator=g) if state else None
    return {n: None if t is None else t.to(DEV) for n, t in d.items()}


def close(got, ref, what, elem, of_max, l2=None):
    g, r = to64(got), np.asarray(ref)
    assert g.shape == r.shape, what
    assert np.isfinite(g).all(), what
    if not r.size:
        return
    err, M = np.abs(g - r), np.abs(r).max()
    assert (err <= elem * np.abs(r) + of_max * M + 1e-30).all(), (what, float(err.max()), float(M))
    if l2 is not None:
        assert np.linalg.norm(g - r) <= l2 * np.linalg.norm(r) + 1e-30, (what, np.linalg.norm(g - r) / np.linalg.norm(r))


def close_state(got, ref, what):
    close(got, ref, what, 0, 2.0 ** -13, 2.0 ** -15)


def close_y(got, ref, what="y"):
    if got.dtype == F32:
        close_state(got, ref, what)
    else:
        close(got, ref, what, 2.0 ** -8, 2.0 ** -10)


def run_and_check(d, out_dtype, scale=0.7):
    y, S = ssm.delta_rule(**d, scale=scale, out_dtype=out_dtype)
    yr, Sr = oracle.delta_rule(**d, scale=scale)
    close_y(y, yr)
    close_state(S, Sr, "final state")
    assert ssm.ssm_device_timeouts() == 0
    return y, S


SHAPES = [  # batch, L, heads, key heads, headdim, dstate
    (1, 1, 1, 1, 8, 8), (2, 2, 2, 1, 16, 24), (1, 31, 3, 3, 24, 32), (2, 32, 4, 2, 64, 64), (1, 33, 4, 1, 32, 128),
    (1, 64, 2, 2, 128, 128), (2, 65, 6, 2, 96, 96), (1, 97, 2, 2, 72, 104), (3, 130, 2, 1, 64, 40), (1, 257, 3, 3, 120, 72),
]


@pytest.mark.parametrize("shape", SHAPES, ids=str)
@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("out", [BF16, F32])
def test_forward(cuda_lib, shape, dtype, out):
    run_and_check(make(*shape, dtype=dtype, seed=sum(shape), state=shape[1] % 2 == 1), out)


def share_misrounded(got, ref):
    """The share of bf16 values that are not the reference's, rounded."""
    return float((got.cpu() != torch.from_numpy(np.ascontiguousarray(ref)).to(BF16)).float().mean())


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_bf16_y_is_the_fp32_result_rounded(cuda_lib, dtype):
    """A bf16 y holds what an fp32 y would, rounded once.  Before the rounding it is off by at
    most d = 2^-15 of its size (relative L2, as an fp32 y).  A value x then rounds the other way
    only where it lies within its error of a border between two steps, which are 2^-8 |x| apart
    or more: a share of at most 2 d |y| / (2^-8 |x|) of the values near x.  Over values spread
    like a normal distribution, E[min(1, 2^-6 / |x|)] with d |y| = 2^-15: 2^-6 0.8 (1 + ln 2^6)
    = 6.4%, and a sixteenth of that at the errors that fp32 sums have.  Operands of 11 bits
    gave 11%."""
    for shape in ((2, 130, 4, 2, 64, 128), (1, 257, 2, 2, 128, 64)):
        d = make(*shape, dtype=dtype, seed=17)
        y, _ = ssm.delta_rule(**d, scale=0.7, out_dtype=BF16)
        assert share_misrounded(y, oracle.delta_rule(**d, scale=0.7)[0]) <= 0.064


def test_forward_many_chunks_long_memory(cuda_lib):
    """1500 tokens whose decay keeps most of the state: errors must not pile up."""
    run_and_check(make(1, 1500, 2, 1, 32, 64, dtype=F32, seed=4, decay=1e-3), F32)


@pytest.mark.parametrize("shape", [(1, 2048, 1, 1, 16, 32), (1, 2101, 2, 1, 32, 64), (2, 3000, 3, 3, 72, 40),
                                   (1, 4255, 2, 2, 128, 128)], ids=str)
@pytest.mark.parametrize("dtype,out", [(BF16, BF16), (F32, F32)])
def test_forward_in_segments(cuda_lib, shape, dtype, out):
    """Long sequences of few heads are cut into segments that run at once; the state is also
    carried in place, which the segments must not race on."""
    d = make(*shape, dtype=dtype, seed=sum(shape), decay=0.02)
    d["a"][:, 700] = -float("inf")
    y, S = run_and_check(d, out)
    state = d["initial_state"].clone()
    y2 = torch.empty_like(y)
    for _ in range(2):
        state.copy_(d["initial_state"])
        ssm.ssm_delta_rule_fwd(**{n: d[n] for n in ("q", "k", "v", "a", "beta")}, y=y2, initial_state=state, final_state=state,
                               scale=0.7)
        assert torch.equal(y2, y) and torch.equal(state, S)
    y0, S0 = ssm.delta_rule(**{**d, "initial_state": None}, scale=0.7, out_dtype=out)
    yr, Sr = oracle.delta_rule(**{**d, "initial_state": None}, scale=0.7)
    close_y(y0, yr)
    close_state(S0, Sr, "final state from zero")


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_forward_hard_gates(cuda_lib, dtype):
    """Full resets (-inf), no decay, growth, steps of 0, 1 and 2, repeated and zero keys."""
    d = make(2, 75, 3, 3, 40, 48, dtype=dtype, seed=9)
    d["a"][:, 10] = d["a"][:, 40, 1] = -float("inf")
    d["a"][:, 20:24] = 0
    d["a"][:, 50] = 0.4
    d["a"][:, 60:62] = -1e30
    d["beta"][:, 5:8] = 0
    d["beta"][:, 30] = 1
    d["beta"][:, 33] = 2
    d["k"][:, 41:46] = d["k"][:, 41:42]
    d["k"][:, 52] = 0
    d["q"][:, 53] = 0
    run_and_check(d, F32)


@pytest.mark.parametrize("kv,st", [(1e8, 1e8), (1e-9, 1e-9), (1e-20, 0.0), (3e4, 1.0)])
def test_forward_any_magnitude(cuda_lib, kv, st):
    """The fp16 operands are scaled: values far outside fp16's range keep their digits."""
    d = make(1, 70, 2, 2, 32, 32, dtype=F32, seed=11)
    d["v"] *= kv
    d["initial_state"] *= st
    run_and_check(d, F32)


def test_forward_any_key_magnitude(cuda_lib):
    """Keys of length 1e-6 and 300, the step scaled so that the recurrence stays stable."""
    for s in (1e-6, 300.0):
        d = make(1, 70, 2, 2, 32, 32, dtype=F32, seed=12)
        d["k"] *= s
        d["q"] *= s
        d["beta"] = d["beta"] / s ** 2
        d["initial_state"] = d["initial_state"] / s
        run_and_check(d, F32, scale=1.0)


def unlike_keys(kind, ratio, dtype, seed=14):
    """Keys whose lengths differ inside a chunk, beta k.k in (0, 1), values of one size.  A
    state that holds what a short key wrote is long / short larger across it: queries are
    unit."""
    d = make(1, 70, 2, 2, 32, 32, dtype=F32, seed=seed)
    g = torch.Generator().manual_seed(seed + 1)
    if kind == "some":
        length = torch.ones(1, 70, 2)
        length[:, ::4] = ratio
    else:
        length = torch.exp(np.log(ratio) / 2 * torch.randn(1, 70, 2, generator=g))
    d["k"] = (d["k"] * length[..., None].to(DEV)).to(dtype)
    d["q"], d["v"] = d["q"].to(dtype), d["v"].to(dtype)
    d["beta"] = (0.1 + 0.8 * torch.rand(1, 70, 2, generator=g)).to(DEV) / (d["k"].float() ** 2).sum(-1)
    return d


UNLIKE = [("some", 30), ("some", 100), ("some", 300), ("lognormal", 30), ("lognormal", 300)]


@pytest.mark.parametrize("kind,ratio", UNLIKE)
@pytest.mark.parametrize("dtype", [BF16, F32])
def test_forward_keys_of_unlike_lengths(cuda_lib, kind, ratio, dtype):
    """Lengths that differ inside a chunk, the step making up for them: the same bounds."""
    run_and_check(unlike_keys(kind, ratio, dtype), F32)


def unlike_rows(shape, dtype, seed=15):
    """Values and states whose rows of headdim differ by up to 2^60."""
    d = make(*shape, dtype=dtype, seed=seed)
    P = shape[4]
    size = 2.0 ** torch.linspace(-30, 30, P)[torch.randperm(P, generator=torch.Generator().manual_seed(seed))].round()
    d["v"] = (d["v"].float() * size.to(DEV)).to(dtype)
    d["initial_state"] = d["initial_state"] * size.to(DEV)[:, None]
    return d


def close_rows(got, ref, what, axis, check=close_state):
    """``check`` row of headdim by row: each against its own size."""
    for i in range(got.shape[axis]):
        check(got.select(axis, i), np.take(ref, i, axis), (what, i))


@pytest.mark.parametrize("shape", [(1, 70, 2, 2, 32, 32), (2, 97, 2, 1, 72, 104), (1, 2101, 2, 1, 32, 64)], ids=str)
@pytest.mark.parametrize("dtype,out", [(BF16, BF16), (F32, F32)])
def test_forward_rows_of_unlike_sizes(cuda_lib, shape, dtype, out):
    """Rows of headdim never meet in the recurrence: each is as exact as if it were alone."""
    d = unlike_rows(shape, dtype)
    y, S = ssm.delta_rule(**d, scale=0.7, out_dtype=out)
    yr, Sr = oracle.delta_rule(**d, scale=0.7)
    close_rows(y, yr, "y", 3, close_y)
    close_rows(S, Sr, "final state", 2)


def bad_rows(shape, dtype):
    """Infinities and NaN in single rows of the start state and of v; the rows they are in."""
    d = make(*shape, dtype=dtype, seed=16)
    d["initial_state"][0, 0, 3, 5] = float("inf")
    d["initial_state"][0, 0, 17, 0] = float("nan")
    d["v"][0, 40, 0, 9] = float("inf")
    d["v"][0, 50, 0, 30] = float("nan")
    clean = {n: t.clone() for n, t in d.items()}
    clean["initial_state"][~clean["initial_state"].isfinite()] = 0
    clean["v"][~clean["v"].isfinite()] = 0
    return d, clean, [3, 9, 17, 30]


@pytest.mark.parametrize("shape", [(1, 70, 2, 2, 32, 32), (1, 2101, 2, 1, 32, 64)], ids=str)
@pytest.mark.parametrize("dtype", [BF16, F32])
def test_forward_bad_rows_stay_alone(cuda_lib, shape, dtype):
    """inf or NaN in a row of the start state or of v reaches that row alone, and there the final
    state and every y from it on; the others keep their bits."""
    d, clean, rows = bad_rows(shape, dtype)
    y, S = ssm.delta_rule(**d, scale=0.7, out_dtype=F32)
    yc, Sc = ssm.delta_rule(**clean, scale=0.7, out_dtype=F32)
    keep = [i for i in range(shape[4]) if i not in rows]
    assert torch.equal(y[:, :, 0][..., keep], yc[:, :, 0][..., keep]) and torch.equal(S[:, 0, keep], Sc[:, 0, keep])
    assert torch.equal(y[:, :, 1], yc[:, :, 1]) and torch.equal(S[:, 1], Sc[:, 1])
    assert not S[:, 0, rows].isfinite().any() and not y[0, :, 0][:, [3, 17]].isfinite().any()
    assert not y[0, 50:, 0][:, rows].isfinite().any()


def test_forward_continues(cuda_lib):
    """A sequence in two calls is the sequence in one, also with the state carried in place."""
    d = make(2, 150, 4, 2, 64, 128, seed=5)
    y, S = ssm.delta_rule(**d, out_dtype=F32)
    cut = {n: d[n][:, :70].contiguous() for n in ("q", "k", "v", "a", "beta")}
    rest = {n: d[n][:, 70:].contiguous() for n in ("q", "k", "v", "a", "beta")}
    state = d["initial_state"].clone()
    for part, at in ((cut, slice(0, 70)), (rest, slice(70, 150))):
        yp = torch.empty_like(part["v"], dtype=F32)
        ssm.ssm_delta_rule_fwd(**part, y=yp, initial_state=state, final_state=state)
        close_state(yp, to64(y[:, at]), "y of the part")
    close_state(state, to64(S), "carried state")


def test_forward_writes_nothing_else(cuda_lib):
    """Guards around y and the final state, a ragged length, and a NaN workspace."""
    d = make(1, 45, 2, 1, 40, 24, seed=6)
    y = torch.full((45 * 2 * 40 + 256,), 7.0, device=DEV, dtype=BF16)
    S = torch.full((2 * 40 * 24 + 128,), 7.0, device=DEV)
    sizes = (1, 45, 2, 1, 40, 24, ssm.SSM_BF16, ssm.SSM_BF16)
    n = ssm.load_library().ssm_delta_rule_fwd_workspace(*sizes)
    ws = torch.full((n // 4 + 64,), float("nan"), device=DEV)
    st = ssm.load_library().ssm_delta_rule_fwd(
        *[d[x].data_ptr() for x in ("q", "k", "v", "a", "beta")], y.data_ptr(), d["initial_state"].data_ptr(), S.data_ptr(),
        1.0, *sizes, ws.data_ptr(), n, torch.cuda.current_stream().cuda_stream)
    assert st == ssm.SSM_OK
    yr, Sr = oracle.delta_rule(**d)
    close_y(y[:3600].reshape(yr.shape), yr)
    close_state(S[:1920].reshape(Sr.shape), Sr, "final state")
    assert bool((y[3600:] == 7).all()) and bool((S[1920:] == 7).all()) and bool(ws[(n + 3) // 4:].isnan().all())


def test_without_workspace_or_final_state(cuda_lib):
    d = make(1, 40, 2, 2, 16, 16, seed=8)
    y = torch.empty_like(d["v"])
    sizes = (1, 40, 2, 2, 16, 16, ssm.SSM_BF16, ssm.SSM_BF16)
    st = ssm.load_library().ssm_delta_rule_fwd(
        *[d[x].data_ptr() for x in ("q", "k", "v", "a", "beta")], y.data_ptr(), d["initial_state"].data_ptr(), None, 1.0,
        *sizes, None, 0, torch.cuda.current_stream().cuda_stream)
    assert st == ssm.SSM_OK
    close_y(y, oracle.delta_rule(**d)[0])


def test_no_tokens(cuda_lib):
    d = make(2, 0, 2, 2, 16, 16)
    y, S = ssm.delta_rule(**d)
    assert y.numel() == 0 and torch.equal(S, d["initial_state"])
    _, S = ssm.delta_rule(**{**d, "initial_state": None})
    assert not S.any()
    dS = torch.randn_like(S)
    g = ssm.delta_rule_bwd(y, **d, dfinal_state=dS)
    assert torch.equal(g["dinitial_state"], dS)


# ---- decode tokens --------------------------------------------------------------------


@pytest.mark.parametrize("shape", [(1, 1, 1, 1, 8, 8), (1, 3, 4, 2, 24, 32), (4, 2, 6, 3, 64, 128), (3, 5, 2, 2, 128, 64),
                                   (7, 33, 3, 1, 40, 96), (2, 2, 2, 2, 16, 104)], ids=str)
@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("out", [BF16, F32])
def test_step(cuda_lib, shape, dtype, out):
    ntok, batch, H, K, P, N = shape
    d = make(batch, ntok, H, K, P, N, dtype=dtype, seed=sum(shape))
    state = d.pop("initial_state")
    yr, Sr = oracle.delta_rule(**d, initial_state=state, scale=0.3)
    t = {n: x.transpose(0, 1).contiguous() for n, x in d.items()}
    one = state.clone()
    y = ssm.delta_rule_step(state, **t, scale=0.3, out_dtype=out)
    elem = 2.0 ** -8 if out == BF16 else 0
    close(y.transpose(0, 1), yr, "y", elem, ntok * 2.0 ** -16)
    close(state, Sr, "state", 0, ntok * 2.0 ** -16)
    # token by token: the same bits (copies: a token's slice need not start on 16 bytes)
    for i in range(ntok):
        yi = ssm.delta_rule_step(one, **{n: x[i:i + 1].clone() for n, x in t.items()}, scale=0.3, out_dtype=out)
        assert torch.equal(yi[0], y[i])
    assert torch.equal(one, state)


def test_prefill_then_decode(cuda_lib):
    """The forward's final state carried through decode tokens is the longer sequence."""
    d = make(2, 60, 4, 2, 64, 128, seed=3, state=False)
    yr, Sr = oracle.delta_rule(**d)
    head = {n: d[n][:, :50].contiguous() for n in ("q", "k", "v", "a", "beta")}
    _, state = ssm.delta_rule(**head)
    tail = {n: d[n][:, 50:].transpose(0, 1).contiguous() for n in ("q", "k", "v", "a", "beta")}
    y = ssm.delta_rule_step(state, **tail, out_dtype=F32)
    close_state(y.transpose(0, 1), yr[:, 50:], "decoded y")
    close_state(state, Sr, "state")


# ---- backward ---------------------------------------------------------------------------


def check_bwd(d, grad_dtype, seed=0, dfinal=True, scale=0.7, of_max=1.0):
    g = torch.Generator().manual_seed(seed)
    dy = torch.randn(d["v"].shape, generator=g).to(DEV).to(grad_dtype)
    b, _, H, P = d["v"].shape
    dS = torch.randn(b, H, P, d["k"].shape[-1], generator=g).to(DEV) if dfinal else None
    got = ssm.delta_rule_bwd(dy, **d, dfinal_state=dS, scale=scale)
    ref = oracle.delta_rule_bwd(dy, **d, dfinal_state=dS, scale=scale)
    for n in ("da", "dbeta"):
        close(got[n], ref[n], n, 0, of_max * 2.0 ** -13, 2.0 ** -14)
    if d["initial_state"] is not None:
        close_state(got["dinitial_state"], ref["dinitial_state"], "dinitial_state")
    else:
        assert got["dinitial_state"] is None
    for n in ("dq", "dk", "dv"):
        assert got[n].dtype == grad_dtype
        if grad_dtype == F32:
            close(got[n], ref[n], n, 0, 2.0 ** -13, 2.0 ** -14)
        else:
            close(got[n], ref[n], n, 2.0 ** -8, 2.0 ** -13 if n == "dv" else 2.0 ** -9)
    assert ssm.ssm_device_timeouts() == 0
    return dy, dS, got


@pytest.mark.parametrize("shape", SHAPES, ids=str)
@pytest.mark.parametrize("dtype,grad", [(BF16, BF16), (F32, F32), (BF16, F32), (F32, BF16)])
def test_backward(cuda_lib, shape, dtype, grad):
    check_bwd(make(*shape, dtype=dtype, seed=sum(shape), state=shape[1] % 2 == 1), grad, seed=1, dfinal=shape[1] % 3 != 0)


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_bf16_gradients_are_the_fp32_results_rounded(cuda_lib, dtype):
    """As a bf16 y: 6.4% of the values round the other way if they are off by 2^-15 before the
    rounding.  The bound is 2%, an error of 2^-17; operands of 11 bits gave 13%."""
    for shape in ((2, 130, 4, 2, 64, 128), (1, 257, 2, 2, 128, 64), (1, 100, 3, 3, 40, 96)):
        d = make(*shape, dtype=dtype, seed=18)
        dy = torch.randn(d["v"].shape, generator=torch.Generator().manual_seed(6)).to(DEV).to(BF16)
        got = ssm.delta_rule_bwd(dy, **d, scale=0.7)
        ref = oracle.delta_rule_bwd(dy, **d, scale=0.7)
        for n in ("dq", "dk", "dv"):
            assert share_misrounded(got[n], ref[n]) <= 0.02, n


def test_backward_long_memory(cuda_lib):
    check_bwd(make(1, 700, 2, 1, 32, 64, dtype=F32, seed=4, decay=1e-3), F32)


@pytest.mark.parametrize("shape", [(1, 2048, 1, 1, 16, 32), (1, 2101, 2, 1, 32, 64), (2, 3000, 3, 3, 72, 40),
                                   (1, 2500, 2, 2, 128, 128)], ids=str)
@pytest.mark.parametrize("dtype,grad", [(BF16, BF16), (F32, F32), (BF16, F32), (F32, BF16)])
def test_backward_in_segments(cuda_lib, shape, dtype, grad):
    """Long sequences of few heads: both passes are cut into segments that run at once."""
    d = make(*shape, dtype=dtype, seed=sum(shape), decay=0.02, state=shape[2] > 1)
    d["a"][:, 700] = -float("inf")
    dy, dS, got = check_bwd(d, grad, seed=2, dfinal=shape[1] != 2101)
    again = ssm.delta_rule_bwd(dy, **d, dfinal_state=dS, scale=0.7)
    assert all(got[n] is None or torch.equal(got[n], again[n]) for n in got)


def test_backward_hard_gates(cuda_lib):
    """beta = 0 (its gradient still counts what would have been written), -inf resets (nothing
    flows past them), repeated and zero keys."""
    d = make(2, 139, 3, 3, 40, 48, dtype=F32, seed=9)
    d["a"][:, 10] = d["a"][:, 64] = -float("inf")
    d["a"][:, 100, 1] = -1e30
    d["a"][:, 20:24] = 0
    d["beta"][:, 5:8] = 0
    d["beta"][:, 30] = 1
    d["k"][:, 41:46] = d["k"][:, 41:42]
    d["k"][:, 52] = 0
    _, _, g = check_bwd(d, F32, seed=2)
    assert float(g["dbeta"][:, 5:8].abs().max()) > 0


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_growing_states(cuda_lib, dtype):
    """Gates above 0 and corrections that overshoot: growth by up to 2^14 within a chunk stays
    within the operands' range, and the bounds are the same."""
    d = make(1, 75, 2, 1, 32, 64, dtype=dtype, seed=21)
    d["a"] = d["a"].abs()                                  # 0 to 0.3: e^4.8 = 2^7 a chunk on average
    run_and_check(d, F32)
    check_bwd(d, F32, seed=4)
    d["a"] = -d["a"]
    d["beta"] = d["beta"] * 2.2
    run_and_check(d, F32)
    check_bwd(d, F32, seed=5)


@pytest.mark.parametrize("kind,ratio", UNLIKE)
@pytest.mark.parametrize("dtype,grad", [(BF16, BF16), (F32, F32)])
def test_backward_keys_of_unlike_lengths(cuda_lib, kind, ratio, dtype, grad):
    check_bwd(unlike_keys(kind, ratio, dtype), grad, seed=6)


@pytest.mark.parametrize("dtype,grad", [(BF16, BF16), (F32, F32)])
def test_backward_rows_of_unlike_sizes(cuda_lib, dtype, grad):
    """The gradients of v and of the start state go row by row, too."""
    d = make(2, 97, 2, 1, 72, 104, dtype=dtype, seed=15)
    g = torch.Generator().manual_seed(7)
    size = (2.0 ** torch.linspace(-30, 30, 72)[torch.randperm(72, generator=g)].round()).to(DEV)
    dy = (torch.randn(d["v"].shape, generator=g).to(DEV) * size).to(grad)
    dS = torch.randn(2, 2, 72, 104, generator=g).to(DEV) * size[:, None]
    got = ssm.delta_rule_bwd(dy, **d, dfinal_state=dS, scale=0.7)
    ref = oracle.delta_rule_bwd(dy, **d, dfinal_state=dS, scale=0.7)
    close_rows(got["dv"], ref["dv"], "dv", 3, close_y)
    close_rows(got["dinitial_state"], ref["dinitial_state"], "dinitial_state", 2)


def sizes_of_da(dy, d, dS, scale):
    """Per token and head the size that da's terms have: |S'| |adjoint of S'|, the norms of the
    two matrices (in 64 bits) whose inner product it is."""
    q, k, v, a, beta = (to64(d[n]) for n in ("q", "k", "v", "a", "beta"))
    H = v.shape[2]
    q, k = (np.repeat(t, H // t.shape[2], 2) for t in (q, k))
    dy, S, mu, dec = to64(dy), to64(d["initial_state"]), to64(dS), []
    for t in range(v.shape[1]):
        S = S * np.exp(a[:, t])[..., None, None]
        dec.append(np.sqrt((S ** 2).sum((-1, -2))))
        e = v[:, t] - np.einsum("bhpn,bhn->bhp", S, k[:, t])
        S = S + (beta[:, t][..., None] * e)[..., None] * k[:, t][..., None, :]
    out = np.empty_like(a)
    for t in reversed(range(v.shape[1])):
        lam = mu + scale * dy[:, t][..., None] * q[:, t][..., None, :]
        de = beta[:, t][..., None] * np.einsum("bhpn,bhn->bhp", lam, k[:, t])
        lam = lam - de[..., None] * k[:, t][..., None, :]
        out[:, t] = np.sqrt((lam ** 2).sum((-1, -2))) * dec[t]
        mu = np.exp(a[:, t])[..., None, None] * lam
    return out


@pytest.mark.parametrize("decay", [0.1, 2, 8, 12, 20, 60])
@pytest.mark.parametrize("dtype,grad", [(BF16, BF16), (F32, F32)])
def test_backward_da_beside_its_own_size(cuda_lib, decay, dtype, grad):
    """da_t is the inner product of S' = exp(a_t) S and its adjoint: off by the products' 2^-13 of
    |S'| |adjoint|, which falls with exp(a_t), not of what the tokens around it have.  Between
    strong decays every term holds one, so the bound is small beside the tensor's largest."""
    d = make(2, 139, 4, 2, 40, 48, dtype=dtype, seed=22)
    d["a"] = -decay * (0.9 + 0.2 * torch.rand(d["a"].shape, generator=torch.Generator().manual_seed(9)).to(DEV))
    d["a"][:, ::9] = -0.01                                 # mild ones between them
    dy, dS, got = check_bwd(d, grad, seed=10)
    ref = oracle.delta_rule_bwd(dy, **d, dfinal_state=dS, scale=0.7)
    err = np.abs(to64(got["da"]) - ref["da"])
    assert (err <= 2.0 ** -13 * sizes_of_da(dy, d, dS, 0.7)).all()


@pytest.mark.parametrize("dtype,grad", [(BF16, BF16), (F32, F32)])
def test_backward_da_at_resets(cuda_lib, dtype, grad):
    """Packed sequences: where exp(a) is 0, da is 0, and a sequence's da does not hold rounding of
    another one's that is 2^13 larger."""
    d = make(1, 200, 2, 1, 64, 64, dtype=dtype, seed=23)
    cuts = [5, 31, 32, 64, 70, 100, 127, 128, 163]
    d["a"][:, cuts] = -INF
    d["a"][:, 100] = -2e4
    for i, (lo, hi) in enumerate(zip([0] + cuts, cuts + [200])):
        if i % 2:
            d["v"][:, lo:hi] *= 2.0 ** 13
    dy, dS, got = check_bwd(d, grad, seed=11)
    ref = oracle.delta_rule_bwd(dy, **d, dfinal_state=dS, scale=0.7)
    assert not got["da"][:, cuts].any()
    err = np.abs(to64(got["da"]) - ref["da"])
    assert (err <= 2.0 ** -13 * sizes_of_da(dy, d, dS, 0.7)).all()


@pytest.mark.parametrize("doublings", [8, 16, 24])
@pytest.mark.parametrize("dtype,grad", [(BF16, BF16), (F32, F32)])
def test_growth_within_a_chunk(cuda_lib, doublings, dtype, grad):
    """States that grow by 2^8, 2^16 and 2^24 within each chunk of 32 tokens.  What a chunk's first
    token adds is by so much larger at its end than what the last one does, and two fp16 pieces
    keep 38 - 24 = 14 bits of the smallest beside the largest: the bounds, relative to the largest
    values, hold."""
    d = make(1, 75, 2, 1, 32, 64, dtype=dtype, seed=24)
    d["a"] = torch.full_like(d["a"], doublings * float(np.log(2)) / 32)
    run_and_check(d, F32)
    check_bwd(d, grad, seed=12)


@pytest.mark.parametrize("dtype,grad", [(BF16, BF16), (F32, F32)])
def test_growth_across_segments(cuda_lib, dtype, grad):
    """A long sequence of few heads whose states grow by 2^20 over each of its segments' 16 chunks
    or more, the segments' maps with them."""
    L = 2101
    d = make(1, L, 2, 1, 32, 64, dtype=dtype, seed=25)
    d["a"] = torch.full_like(d["a"], 20 * float(np.log(2)) / 512)
    run_and_check(d, F32)
    check_bwd(d, grad, seed=13)


def test_backward_tiny_gradients(cuda_lib):
    """Gradients of 1e-9, as behind a mean over a large batch: the scaled operands keep them."""
    d = make(1, 90, 2, 2, 64, 64, seed=13)
    dy, _, g = check_bwd(d, BF16, seed=3, dfinal=False)
    small = ssm.delta_rule_bwd((dy.float() * 2.0 ** -30).to(BF16), **d, scale=0.7)
    for n in ("dq", "dk", "dv", "da", "dbeta"):
        assert torch.equal(small[n].float() * 2.0 ** 30, g[n].float()), n    # powers of two: the same digits


def test_backward_by_differences(cuda_lib):
    """Directional derivatives of the GPU's own fp32 forward against its gradients."""
    d = make(1, 40, 2, 1, 16, 16, dtype=F32, seed=21)
    dy, dS, g = check_bwd(d, F32, seed=4)
    w = {n: torch.randn(t.shape, generator=torch.Generator().manual_seed(5)).to(DEV) for n, t in d.items()}

    def loss(h):
        y, S = ssm.delta_rule(**{n: t + h * w[n] for n, t in d.items()}, scale=0.7)
        return float((dy.double() * y.double()).sum() + (dS.double() * S.double()).sum())

    want = sum(float((g["d" + n].double() * w[n].double()).sum()) for n in d)
    # central difference: h^2 f''' / 6 (h = 2^-7: 1e-5 of third derivatives of order 10 want) and
    # fp32 noise of y, 2^-15 of the summands' size, over 2h
    h = 2.0 ** -7
    noise = 2.0 ** -15 * float(dy.double().norm() * 3) / (2 * h)
    assert abs((loss(h) - loss(-h)) / (2 * h) - want) <= 2e-3 * abs(want) + noise + 0.05


def test_results_do_not_vary(cuda_lib):
    d = make(3, 333, 6, 3, 64, 128, seed=7)
    dy = torch.randn(d["v"].shape, device=DEV).to(BF16)
    y, S = ssm.delta_rule(**d)
    g = ssm.delta_rule_bwd(dy, **d)
    for _ in range(3):
        y2, S2 = ssm.delta_rule(**d)
        g2 = ssm.delta_rule_bwd(dy, **d)
        assert torch.equal(y, y2) and torch.equal(S, S2)
        assert all(torch.equal(g[n], g2[n]) for n in g)


# ---- values that are not finite --------------------------------------------------------------


def right_or_not_finite(got, ref, what, elem, of_max):
    """Where a result is finite it is the right one."""
    g, r = to64(got), np.asarray(ref)
    ok, M = np.isfinite(g), np.abs(r[np.isfinite(r)]).max(initial=0)
    with np.errstate(invalid="ignore"):
        assert (np.abs(g - r)[ok] <= elem * np.abs(r[ok]) + of_max * M).all(), what


BAD = [(n, t, x) for n in ("q", "k", "v", "beta", "a") for t in (52, 40, 75) for x in (INF, NAN)] + [
    ("initial_state", 3, INF), ("initial_state", 3, NAN)]


def with_bad(name, at, value, dtype):
    d = make(1, 150, 2, 2, 40, 48, dtype=dtype, seed=19)
    d[name][(0, 0, at, 5) if name == "initial_state" else (0, at, 0) + (7,) * (d[name].dim() - 3)] = value
    return d


@pytest.mark.parametrize("name,at,value", BAD)
@pytest.mark.parametrize("dtype", [BF16, F32])
def test_forward_not_finite(cuda_lib, name, at, value, dtype):
    """An inf or NaN anywhere: what comes out finite is right, and chunks of 32 tokens before it
    and the other head come out as without it."""
    d = with_bad(name, at, value, dtype)
    y, S = ssm.delta_rule(**d, scale=0.7, out_dtype=F32)
    with np.errstate(invalid="ignore", over="ignore"):
        yr, Sr = oracle.delta_rule(**d, scale=0.7)
    right_or_not_finite(y, yr, "y", 0, 2.0 ** -13)
    right_or_not_finite(S, Sr, "final state", 0, 2.0 ** -13)
    before = 0 if name == "initial_state" else at // 32 * 32
    assert y[:, :before].isfinite().all() and y[:, :, 1].isfinite().all() and S[:, 1].isfinite().all()


@pytest.mark.parametrize("name,at,value", BAD + [
    ("dy", 52, INF), ("dy", 40, NAN), ("dfinal_state", 3, INF), ("dfinal_state", 3, NAN)])
@pytest.mark.parametrize("dtype,grad", [(BF16, BF16), (F32, F32)])
def test_backward_not_finite(cuda_lib, name, at, value, dtype, grad):
    ours = name not in ("dy", "dfinal_state")
    d = with_bad(name, at, value, dtype) if ours else make(1, 150, 2, 2, 40, 48, dtype=dtype, seed=19)
    g = torch.Generator().manual_seed(8)
    more = dict(dy=torch.randn(d["v"].shape, generator=g).to(DEV).to(grad),
                dfinal_state=torch.randn(1, 2, 40, 48, generator=g).to(DEV))
    if not ours:
        more[name][(0, at, 0, 7) if name == "dy" else (0, 0, at, 5)] = value
    got = ssm.delta_rule_bwd(more["dy"], **d, dfinal_state=more["dfinal_state"], scale=0.7)
    with np.errstate(invalid="ignore", over="ignore"):
        ref = oracle.delta_rule_bwd(more["dy"], **d, dfinal_state=more["dfinal_state"], scale=0.7)
    for n in got:
        right_or_not_finite(got[n], ref[n], n, 2.0 ** -8 if got[n].dtype == BF16 else 0, 2.0 ** -12)
        assert (got[n][:, 1] if n == "dinitial_state" else got[n][:, :, 1]).isfinite().all(), n


@pytest.mark.parametrize("name,value", [(n, x) for n in ("q", "k", "v", "beta", "a", "initial_state") for x in (INF, NAN)])
def test_not_finite_in_segments(cuda_lib, name, value):
    """The same in a long sequence whose segments run at once, with their maps."""
    d = make(1, 2101, 2, 1, 32, 64, dtype=F32, seed=26, decay=0.02)
    at = (0, 0, 3, 5) if name == "initial_state" else (0, 1200, 0) + (7,) * (d[name].dim() - 3)
    d[name][at] = value
    dy = torch.randn(d["v"].shape, generator=torch.Generator().manual_seed(14)).to(DEV)
    y, S = ssm.delta_rule(**d, scale=0.7)
    got = ssm.delta_rule_bwd(dy, **d, scale=0.7)
    with np.errstate(invalid="ignore", over="ignore"):
        yr, Sr = oracle.delta_rule(**d, scale=0.7)
        ref = oracle.delta_rule_bwd(dy, **d, scale=0.7)
    right_or_not_finite(y, yr, "y", 0, 2.0 ** -13)
    right_or_not_finite(S, Sr, "final state", 0, 2.0 ** -13)
    for n in got:
        right_or_not_finite(got[n], ref[n], n, 0, 2.0 ** -12)
    if name != "initial_state":
        assert y[:, :1184].isfinite().all()


# ---- streams and graphs --------------------------------------------------------------------


def test_two_streams_at_once(cuda_lib):
    ds = [make(2, 200, 4, 2, 64, 64, seed=30 + i) for i in range(2)]
    want = [ssm.delta_rule(**d) for d in ds]
    dy = torch.ones_like(ds[0]["v"])
    wantg = [ssm.delta_rule_bwd(dy, **d) for d in ds]
    torch.cuda.synchronize()
    streams, got = [torch.cuda.Stream() for _ in range(2)], [[], []]
    for _ in range(4):
        for i, s in enumerate(streams):
            with torch.cuda.stream(s):
                got[i].append((ssm.delta_rule(**ds[i]), ssm.delta_rule_bwd(dy, **ds[i])))
    torch.cuda.synchronize()
    for i in range(2):
        for (y, S), g in got[i]:
            assert torch.equal(y, want[i][0]) and torch.equal(S, want[i][1])
            assert all(torch.equal(g[n], wantg[i][n]) for n in g)


def test_stream_argument(cuda_lib):
    """The call runs, scratch included, on the stream that it is given."""
    d = make(1, 120, 2, 2, 64, 64, seed=40)
    want, _ = ssm.delta_rule(**d)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    y, S = torch.empty_like(d["v"]), torch.empty_like(d["initial_state"])
    ssm.ssm_delta_rule_fwd(**{n: d[n] for n in ("q", "k", "v", "a", "beta")}, y=y, initial_state=d["initial_state"],
                           final_state=S, stream=s)
    s.synchronize()
    assert torch.equal(y, want)


def test_captured_and_replayed(cuda_lib):
    """Forward, backward and decode tokens in two graphs, replayed in turn on new inputs."""
    d = make(2, 100, 4, 2, 64, 64, seed=50)
    dy = torch.randn(d["v"].shape, device=DEV).to(BF16)
    state = torch.zeros(2, 4, 64, 64, device=DEV)
    t = {n: d[n][:, :2].transpose(0, 1).contiguous() for n in ("q", "k", "v", "a", "beta")}

    def all_calls():
        return ssm.delta_rule(**d), ssm.delta_rule_bwd(dy, **d), ssm.delta_rule_step(state, **t)

    all_calls()
    torch.cuda.synchronize()
    graphs, outs = [], []
    for _ in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(all_calls())
        graphs.append(g)
    for i in range(4):
        new = make(2, 100, 4, 2, 64, 64, seed=60 + i)
        for n in ("q", "k", "v", "a", "beta", "initial_state"):
            d[n].copy_(new[n])
        state.zero_()
        graphs[i % 2].replay()
        (y, S), g, ys = (x for x in outs[i % 2])
        got = [y.clone(), S.clone(), *(g[n].clone() for n in sorted(g)), ys.clone(), state.clone()]
        state.zero_()
        (y, S), g, ys = all_calls()
        want = [y, S, *(g[n] for n in sorted(g)), ys, state]
        assert all(torch.equal(a, b) for a, b in zip(got, want))
    del graphs


def test_offsets_past_32_bits(cuda_lib):
    """More than 2^31 values (2^32 bytes) before the last sequence's rows."""
    b, L, H, P, N = 65, 4096, 64, 128, 8
    g = torch.Generator(device=DEV).manual_seed(1)
    v = torch.zeros(b, L, H, P, device=DEV, dtype=BF16)
    assert v.numel() > 2 ** 31
    q, k = (torch.zeros(b, L, 1, N, device=DEV, dtype=BF16) for _ in range(2))
    a, beta = torch.zeros(b, L, H, device=DEV), torch.zeros(b, L, H, device=DEV)
    last = make(1, 64, H, 1, P, N, seed=2)
    for t, n in ((v, "v"), (q, "q"), (k, "k"), (a, "a"), (beta, "beta")):
        t[-1, -64:] = last[n][0]
    y, S = ssm.delta_rule(q, k, v, a, beta)
    yr, Sr = oracle.delta_rule(**{n: last[n] for n in ("q", "k", "v", "a", "beta")})
    close_y(y[-1:, -64:], yr)
    close_state(S[-1:], Sr, "final state")
    assert not y[0].any()
    del g
