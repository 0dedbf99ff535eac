"""Host-side checks of the delta rule's and the layer norm's entry points: what is refused,
with which status, before anything is launched (fake device addresses, no GPU)."""
import pytest
import torch

import selective_state_space_45_b200 as ssm
from selective_state_space_45_b200 import build as ssm_build

INV, UNS, ALI, SCR, OK = (ssm.SSM_ERR_INVALID_ARG, ssm.SSM_ERR_UNSUPPORTED, ssm.SSM_ERR_ALIGNMENT, ssm.SSM_ERR_SCRATCH,
                          ssm.SSM_OK)
# distinct fake buffers, 16 MiB apart
BUF = [0x7F0000000000 + k * (1 << 24) for k in range(20)]
Q, KK, V, A, B, Y, H0, H1, DY, DF, DQ, DK, DV, DA, DB, DH, WS = BUF[:17]


@pytest.fixture(scope="module")
def lib():
    ssm_build.build()
    return ssm.load_library()


SIZES = dict(batch=2, L=8, H=4, K=2, P=64, N=128, din=ssm.SSM_BF16, dout=ssm.SSM_BF16)


def _sizes(a):
    return [a[n] for n in ("batch", "L", "H", "K", "P", "N", "din", "dout")]


def fwd(lib, **kw):
    a = dict(q=Q, k=KK, v=V, a=A, beta=B, y=Y, h0=H0, h1=H1, ws=WS, nws=1 << 23, **SIZES)
    a.update(kw)
    return lib.ssm_delta_rule_fwd(*[a[n] for n in ("q", "k", "v", "a", "beta", "y", "h0", "h1")], 1.0, *_sizes(a),
                                  a["ws"], a["nws"], None)


def step(lib, **kw):
    a = dict(state=H0, q=Q, k=KK, v=V, a=A, beta=B, y=Y, **SIZES)
    a.update(kw)
    s = _sizes(a)
    return lib.ssm_delta_rule_step(*[a[n] for n in ("state", "q", "k", "v", "a", "beta", "y")], 1.0, s[1], s[0], *s[2:],
                                   None)


def bwd(lib, **kw):
    a = dict(q=Q, k=KK, v=V, a=A, beta=B, h0=H0, dy=DY, df=DF, dq=DQ, dk=DK, dv=DV, da=DA, db=DB, dh=DH, ws=WS,
             nws=1 << 23, **SIZES)
    a.update(kw)
    return lib.ssm_delta_rule_bwd(*[a[n] for n in ("q", "k", "v", "a", "beta", "h0", "dy", "df", "dq", "dk", "dv", "da",
                                                   "db", "dh")], 1.0, *_sizes(a), a["ws"], a["nws"], None)


SIZE_REFUSALS = [
    (dict(batch=-1), INV), (dict(L=-1), INV), (dict(H=-4), INV), (dict(K=-2), INV),
    (dict(H=4, K=3), INV), (dict(H=2, K=4), INV), (dict(K=0), INV),          # key heads that do not divide the heads
    (dict(P=0), INV), (dict(N=0), INV), (dict(P=12), UNS), (dict(N=20), UNS), (dict(P=136), UNS), (dict(N=256), UNS),
    (dict(din=2), INV), (dict(dout=-1), INV), (dict(L=2 ** 31 - 1), UNS),
]


@pytest.mark.parametrize("kw,status", SIZE_REFUSALS)
def test_sizes_are_refused_alike(lib, kw, status):
    assert fwd(lib, **kw) == status
    assert step(lib, **kw) == status
    assert bwd(lib, **kw) == status
    s = _sizes({**SIZES, **kw})
    assert lib.ssm_delta_rule_fwd_workspace(*s) == 0 and lib.ssm_delta_rule_bwd_workspace(*s) == 0


@pytest.mark.parametrize("kw,status", [
    (dict(q=None), INV), (dict(k=None), INV), (dict(v=None), INV), (dict(a=None), INV), (dict(beta=None), INV),
    (dict(y=None), INV), (dict(q=Q + 8), ALI), (dict(h0=H0 + 4), ALI), (dict(h1=H1 + 8), ALI), (dict(ws=WS + 8), ALI),
    (dict(y=V), INV), (dict(y=H0), INV), (dict(h1=KK), INV), (dict(h1=H0 + 64), INV),      # overlaps
    (dict(ws=Y), INV), (dict(ws=Q + 16), INV), (dict(ws=H1), INV),
    (dict(nws=64), SCR),
    (dict(batch=0), OK), (dict(H=0, K=0), OK), (dict(L=0, h1=None), OK), (dict(L=0, h0=H1), OK),
])
def test_forward_refusals(lib, kw, status):
    assert fwd(lib, **kw) == status


@pytest.mark.parametrize("kw,status", [
    (dict(state=None), INV), (dict(q=None), INV), (dict(y=None), INV), (dict(state=H0 + 4), ALI), (dict(a=A + 4), ALI),
    (dict(y=H0), INV), (dict(state=V), INV), (dict(y=B), INV), (dict(L=0, state=None), OK), (dict(batch=0), OK),
])
def test_step_refusals(lib, kw, status):
    assert step(lib, **kw) == status


@pytest.mark.parametrize("kw,status", [
    (dict(dy=None), INV), (dict(dq=None), INV), (dict(dk=None), INV), (dict(dv=None), INV), (dict(da=None), INV),
    (dict(db=None), INV), (dict(q=None), INV), (dict(beta=None), INV), (dict(dy=DY + 2), ALI), (dict(dh=DH + 4), ALI),
    (dict(dv=DY), INV), (dict(dq=DK), INV), (dict(da=DB), INV), (dict(dh=DF), INV), (dict(ws=DQ), INV), (dict(ws=DY), INV),
    (dict(ws=WS + 8), ALI), (dict(nws=1024), SCR), (dict(batch=0), OK), (dict(L=0, dh=None), OK),
])
def test_backward_refusals(lib, kw, status):
    assert bwd(lib, **kw) == status


def ln_fwd(lib, **kw):
    a = dict(x=Q, w=A, b=B, y=Y, mean=DA, rstd=DB, eps=1e-5, rows=8, dim=64, din=ssm.SSM_BF16, dout=ssm.SSM_F32)
    a.update(kw)
    return lib.ssm_layer_norm_fwd(*[a[n] for n in ("x", "w", "b", "y", "mean", "rstd", "eps", "rows", "dim", "din", "dout")],
                                  None)


def ln_bwd(lib, **kw):
    a = dict(dy=DY, x=Q, w=A, mean=DA, rstd=DB, dx=DQ, dw=DK, db=DV, rows=8, dim=64, din=ssm.SSM_BF16, dout=ssm.SSM_F32,
             ws=WS, nws=1 << 20)
    a.update(kw)
    return lib.ssm_layer_norm_bwd(*[a[n] for n in ("dy", "x", "w", "mean", "rstd", "dx", "dw", "db", "rows", "dim", "din",
                                                   "dout", "ws", "nws")], None)


@pytest.mark.parametrize("kw,status", [
    (dict(rows=-1), INV), (dict(dim=0), INV), (dict(dim=8193), UNS), (dict(din=5), INV), (dict(dout=2), INV),
])
def test_norm_sizes_are_refused_alike(lib, kw, status):
    assert ln_fwd(lib, **kw) == status
    assert ln_bwd(lib, **kw) == status


@pytest.mark.parametrize("kw,status", [
    (dict(x=None), INV), (dict(y=None), INV), (dict(eps=-1e-5), INV), (dict(eps=float("nan")), INV), (dict(x=Q + 2), ALI),
    (dict(w=A + 4), ALI), (dict(mean=DA + 4), ALI), (dict(y=Q), INV), (dict(mean=DB), INV), (dict(rstd=A), INV),
    (dict(rows=0, x=None, y=None), OK),
])
def test_norm_forward_refusals(lib, kw, status):
    assert ln_fwd(lib, **kw) == status


@pytest.mark.parametrize("kw,status", [
    (dict(dy=None), INV), (dict(x=None), INV), (dict(mean=None), INV), (dict(rstd=None), INV), (dict(dx=None), INV),
    (dict(dx=DY), INV), (dict(dw=A), INV), (dict(dw=DV), INV), (dict(ws=DQ), INV), (dict(ws=Q), INV), (dict(dx=DQ + 4), ALI),
    (dict(ws=WS + 4), ALI), (dict(nws=16), SCR),
])
def test_norm_backward_refusals(lib, kw, status):
    assert ln_bwd(lib, **kw) == status


def test_binding_refuses_before_the_library():
    """Wrong shapes, dtypes, strides and devices raise ValueError in the binding."""
    def t(*s, dtype=torch.float32):
        return torch.zeros(s, dtype=dtype)

    good = dict(q=t(1, 4, 2, 8), k=t(1, 4, 2, 8), v=t(1, 4, 2, 8), a=t(1, 4, 2), beta=t(1, 4, 2))
    for name, bad in (("k", t(1, 4, 2, 16)), ("a", t(1, 4, 2, dtype=torch.bfloat16)), ("beta", t(1, 3, 2)),
                      ("q", t(1, 4, 2, 8, dtype=torch.bfloat16)), ("v", t(4, 2, 8)), ("k", t(1, 4, 8, 2).transpose(2, 3))):
        with pytest.raises(ValueError):
            ssm.delta_rule(**{**good, name: bad})
    with pytest.raises(ValueError, match="CUDA"):
        ssm.delta_rule(**good)
    with pytest.raises(ValueError):
        ssm.delta_rule_step(t(2, 2, 8, 8), **good)               # a state of another batch
    with pytest.raises(ValueError):
        ssm.delta_rule_bwd(t(1, 4, 2, 16), **good)
    x = t(4, 8)
    for args in ((x, t(7)), (x, t(8, dtype=torch.bfloat16)), (x.t(), t(4))):
        with pytest.raises(ValueError):
            ssm.layer_norm(*args)
    with pytest.raises(ValueError):
        ssm.layer_norm_bwd(x, x, None, t(3), t(4))


@pytest.mark.parametrize("rows", [2 ** 31, 2 ** 32, 2 ** 32 + 8])
def test_norm_rows_past_32_bits_are_refused(monkeypatch, rows):
    """A count of rows that the library's int does not hold raises; nothing is called with what is
    left of it."""
    from selective_state_space_45_b200 import _lib

    called = []
    monkeypatch.setattr(_lib, "_require", lambda shapes: None)
    monkeypatch.setattr(_lib, "_call_on", lambda *a, **k: called.append(a))
    x = torch.empty(rows, 8, dtype=torch.bfloat16, device="meta")
    s = torch.empty(rows, device="meta")
    monkeypatch.setattr(_lib, "_at", lambda t: None)
    for call in (lambda: ssm.layer_norm(x), lambda: ssm.ssm_layer_norm_fwd(x, None, None, x),
                 lambda: ssm.layer_norm_bwd(x, x, None, s, s), lambda: ssm.ssm_layer_norm_bwd(x, x, None, s, s, x)):
        with pytest.raises(ValueError, match="rows: at most"):
            call()
    assert not called


def test_sizes_past_32_bits_are_refused(monkeypatch):
    """The same for the lengths of the scan, the convolution and their decode forms."""
    from selective_state_space_45_b200 import _lib

    class Never:
        def __getattr__(self, name):
            raise AssertionError(name + " was called")

    monkeypatch.setattr(_lib, "load_library", Never)
    L = 2 ** 32
    bf = dict(dtype=torch.bfloat16, device="meta")
    x, B, h = torch.empty(1, 1, L, **bf), torch.empty(1, L, 1, **bf), torch.empty(L, 1, 1, device="meta")
    A, xb, Bb = torch.empty(1, 1, device="meta"), torch.empty(L, 1, **bf), torch.empty(L, 1, **bf)
    xs, Bs, a = torch.empty(1, L, 1, 32, **bf), torch.empty(1, L, 1, 64, **bf), torch.empty(1, L, 1, device="meta")
    for call in (lambda: ssm.selective_scan(x, x, A, B, B), lambda: ssm.selective_scan_bwd(x, x, x, A, B, B),
                 lambda: ssm.ssm_selective_scan_fwd(x, x, None, 0, A, B, B, None, None, x, None),
                 lambda: ssm.ssm_selective_scan_fwd_noalloc(x, x, None, 0, A, B, B, None, None, x, None),
                 lambda: ssm.ssm_state_step(h, xb, xb, A, Bb, Bb, None, None, xb),
                 lambda: ssm.ssm_state_step_multi(h, xb[None], xb[None], A, Bb[None], Bb[None], None, None, xb[None]),
                 lambda: ssm.causal_conv1d(x, A), lambda: ssm.ssm_causal_conv1d_step(None, xb, A, None, xb),
                 lambda: ssm.ssd(xs, a, Bs, Bs)):
        with pytest.raises(ValueError, match="2\\^31"):
            call()


def test_scratch_status_names_both_causes():
    ssm_build.build()
    text = ssm.ssm_status_string(SCR)
    assert "workspace" in text and "allocation-free" in text


@pytest.mark.parametrize("kw", [dict(batch=8, L=2048, H=24, K=24), dict(batch=3, L=1021, H=8, K=4, P=128, N=64, din=0, dout=0),
                                dict(batch=8, L=2048, H=24, K=24, P=64, N=64, din=0, dout=0), dict(batch=2, L=4096, H=48, K=48, P=8)])
def test_scratch_is_what_the_header_says(lib, kw):
    """The sums that include/ssm.h states, for sizes that are not cut into segments: within 5%
    above for the rest (a few values per chunk, a chunk's and a span's ends)."""
    a = {**SIZES, **kw}
    tok, P, N = a["batch"] * a["L"], -(-a["P"] // 64) * 64, -(-a["N"] // 32) * 32
    rows = a["K"] * (4 * N + 32) * (2 if a["din"] == ssm.SSM_F32 else 1)
    bwd = a["H"] * (224 + (12 if a["dout"] == ssm.SSM_F32 else 10) * P + P * N / 8) + rows
    bwd += 8 * a["N"] * a["K"] if a["H"] > a["K"] else 0
    for got, want in ((lib.ssm_delta_rule_fwd_workspace(*_sizes(a)), tok * (224 * a["H"] + rows)),
                      (lib.ssm_delta_rule_bwd_workspace(*_sizes(a)), tok * bwd)):
        assert want <= got <= 1.05 * want


def test_a_stream_of_another_device_is_refused(monkeypatch):
    """The call would run on another stream than the given one."""
    from selective_state_space_45_b200 import _lib

    class On:
        is_cuda, device = True, torch.device("cuda", 1)

    class Stream:
        device = torch.device("cuda", 0)

    monkeypatch.setattr(torch.cuda, "Stream", Stream)
    with pytest.raises(ValueError, match="stream of cuda:0"):
        _lib._current(Stream(), On)
