"""Calls that are given a stream: what they allocate belongs to that stream, so that its memory
is not handed out again, nor was in use, by another one."""
import pytest
import torch

import selective_state_space_45_b200 as ssm

pytestmark = pytest.mark.gpu
DEV = "cuda"


def calls():
    """Every call of the binding that allocates, as f(stream) -> tensors."""
    g = torch.Generator().manual_seed(3)

    def n(*s, dtype=torch.bfloat16):
        return torch.randn(s, generator=g).to(DEV).to(dtype)

    f32 = torch.float32
    x, dl, z, dy = (n(2, 32, 40) for _ in range(4))
    dl = torch.nn.functional.softplus(dl)
    A, D, B, C = -n(32, 16, dtype=f32).abs(), n(32, dtype=f32), n(2, 40, 16), n(2, 40, 16)
    w = n(32, 4, dtype=f32)
    xs, Bs, Cs, as_ = n(1, 40, 2, 64), n(1, 40, 2, 64), n(1, 40, 2, 64), -n(1, 40, 2, dtype=f32).abs()
    q, k = (torch.nn.functional.normalize(n(1, 40, 2, 64).float(), dim=-1).to(torch.bfloat16) for _ in range(2))
    d = dict(q=q, k=k, v=n(1, 40, 2, 64), a=-n(1, 40, 2, dtype=f32).abs(), beta=torch.sigmoid(n(1, 40, 2, dtype=f32)))
    h0 = n(1, 2, 64, 64, dtype=f32)
    r, wn, bn = n(64, 96), n(96, dtype=f32), n(96, dtype=f32)
    _, mean, rstd = ssm.layer_norm(r, wn, bn, return_stats=True)
    kept = []

    def step(s):
        kept.append(h0.repeat(40, 1, 1, 1))                # updated in place: there before the call, and until its end
        torch.cuda.synchronize()
        return ssm.delta_rule_step(kept[-1], **d, stream=s)

    return {
        "selective_scan": lambda s: ssm.selective_scan(x, dl, A, B, C, D=D, z=z, stream=s),
        "selective_scan_bwd": lambda s: ssm.selective_scan_bwd(dy, x, dl, A, B, C, D=D, z=z, stream=s),
        "causal_conv1d": lambda s: ssm.causal_conv1d(x, w, return_final_window=True, stream=s),
        "ssd": lambda s: ssm.ssd(xs, as_, Bs, Cs, stream=s),
        "delta_rule": lambda s: ssm.delta_rule(**d, initial_state=h0, stream=s),
        "delta_rule_step": step,
        "delta_rule_bwd": lambda s: ssm.delta_rule_bwd(d["v"], **d, initial_state=h0, stream=s),
        "layer_norm": lambda s: ssm.layer_norm(r, wn, bn, return_stats=True, stream=s),
        "layer_norm_bwd": lambda s: ssm.layer_norm_bwd(r, r, wn, mean, rstd, stream=s),
    }


NAMES = ("selective_scan", "selective_scan_bwd", "causal_conv1d", "ssd", "delta_rule", "delta_rule_step", "delta_rule_bwd",
         "layer_norm", "layer_norm_bwd")


def tensors(out):
    out = out.values() if isinstance(out, dict) else out if isinstance(out, tuple) else (out,)
    return [t for t in out if t is not None]


def stream_of(t):
    """The stream whose pool a tensor's memory is of."""
    for seg in torch.cuda.memory_snapshot():
        if seg["address"] <= t.data_ptr() < seg["address"] + seg["total_size"]:
            return seg["stream"]
    raise AssertionError("not of torch's allocator")


@pytest.mark.parametrize("name", NAMES)
@pytest.mark.parametrize("how", ["object", "handle"])
def test_outputs_are_of_the_calls_stream(cuda_lib, name, how):
    call = calls()[name]
    want = tensors(call(None))
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    got = tensors(call(s if how == "object" else s.cuda_stream))
    s.synchronize()
    assert all(stream_of(t) == s.cuda_stream for t in got)
    assert all(torch.equal(a, b) for a, b in zip(got, want))


@pytest.mark.parametrize("name", NAMES)
def test_the_default_stream_given_from_another(cuda_lib, name):
    call = calls()[name]
    want = tensors(call(None))
    torch.cuda.synchronize()
    default = torch.cuda.default_stream()
    with torch.cuda.stream(torch.cuda.Stream()):
        by_object, by_handle = tensors(call(default)), tensors(call(0))
    torch.cuda.synchronize()
    for got in (by_object, by_handle):
        assert all(stream_of(t) == 0 for t in got)
        assert all(torch.equal(a, b) for a, b in zip(got, want))
