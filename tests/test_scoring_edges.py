"""The scoring path's edges that need no GPU: the oracle's exact e4m3 quotients
and what the Python layer refuses."""

from __future__ import annotations

from fractions import Fraction

import numpy as np
import pytest
import torch

import lm_head_projection_b200 as pkg
from oracle import scoring_oracle as o

no_gpu = pytest.mark.skipif(torch.cuda.is_available(),
                            reason="placeholder pointers must not reach a real device")
P = 4096  # placeholder, 16-byte aligned, never dereferenced


def _nearest_e4m3(q: Fraction) -> float:
    """The nearest e4m3 number to a fraction in [-448, 448], by trying them all."""
    every = [Fraction(k, 512) for k in range(8)]
    every += [Fraction(8 + k) * Fraction(2) ** (e - 3) for e in range(-6, 9) for k in range(8)]
    every = [f for f in every if f <= 448]
    a = abs(q)
    d = [abs(f - a) for f in every]
    i = min(range(len(every)), key=lambda j: (d[j], j % 2))  # (the j-th has the code j)
    return float(every[i]) * (-1 if q < 0 else 1)


def test_exact_quotients_against_fractions():
    rs = np.random.RandomState(0)
    m = rs.randint(128, 256, 3000) * 2.0 ** rs.randint(-20, 20, 3000)
    v = np.minimum(rs.randint(128, 256, 3000) * 2.0 ** rs.randint(-16, 1, 3000) / 256, 1)
    v = np.where(v * m <= m, np.round(v * 256) / 256 * 2.0 ** rs.randint(-16, 1, 3000), 1.0)
    v = v * 2.0 ** np.floor(np.log2(m)) * rs.choice([-1, 1], 3000)
    v[:200] = m[:200] * rs.choice([1.0, 0.5, 15 / 16, 31 / 32, 2.0 ** -18, 0.0], 200)
    got = o.e4m3_quotients(v, m)
    for x, d, g in zip(v, m, got):
        assert g == _nearest_e4m3(448 * Fraction(float(x)) / Fraction(float(d))), (x, d)
    # ties go to even: 17 / 448 of the largest lies between codes 16 and 18
    assert o.e4m3_quotients(17.0, 448.0) == 16 and o.e4m3_quotients(-19.0, 448.0) == -20


@no_gpu
def test_wait_selftest_refusals():
    f = lambda role=1, ms=20, K=64, D=P: pkg.flkl_fp8_wait_selftest(P, P, P, P, 4, 8, K, D, role,
                                                                   0, ms, 0)
    assert f(role=0) == 1 and f(role=4) == 1 and f(ms=0) == 1 and f(ms=1001) == 1
    assert f(K=24) == 2 and f(D=0) == 1


def test_overwriting_what_requires_a_gradient_is_refused():
    """Before anything is launched, and only while gradients are recorded."""
    from lm_head_projection_b200 import fp8, norm

    x, w = torch.zeros(4, 64), torch.ones(64)
    r = torch.zeros(4, 64, requires_grad=True)
    with pytest.raises(ValueError, match="requires a gradient"):
        norm.add_rms_norm(x, w, r, inplace=True)
    q = torch.zeros(4, 64, dtype=torch.float8_e4m3fn)
    s1, s2 = torch.ones(4, 1), torch.ones(1, 1)
    d = torch.zeros(4, 4, requires_grad=True)
    with pytest.raises(ValueError, match="requires a gradient"):
        fp8.block_matmul(q, s1, q, s2, out_dtype=torch.float32, out=d)
    with torch.no_grad(), pytest.raises(ValueError, match="CUDA"):
        norm.add_rms_norm(x, w, r, inplace=True)
    with torch.no_grad(), pytest.raises(ValueError, match="CUDA"):
        fp8.block_matmul(q, s1, q, s2, out_dtype=torch.float32, out=d)


def _cpu_head(monkeypatch, bias=True):
    """A head whose codes a stand-in for the quantiser made, since there is no GPU."""
    from lm_head_projection_b200 import fp8

    g = torch.Generator().manual_seed(1)
    codes = torch.randn(256, 64, generator=g).to(torch.float8_e4m3fn)
    scale = torch.rand(2, 1, generator=g) + 0.1
    monkeypatch.setattr(fp8, "quantize_blocks", lambda w, stream=None: (codes, scale))
    b = torch.randn(256, generator=g) if bias else None
    return fp8.Fp8Head(torch.zeros(256, 64), b), codes, scale, b


@pytest.mark.parametrize("cast", [
    lambda m: m.to(torch.bfloat16), lambda m: m.half(), lambda m: m.double(),
    lambda m: m.float(), lambda m: m.bfloat16(), lambda m: m.to("cpu", torch.float16),
    lambda m: m.to(torch.zeros(1, dtype=torch.bfloat16)), lambda m: m.cpu()])
@pytest.mark.parametrize("bias", [True, False])
def test_a_head_keeps_its_types_under_a_cast_of_the_model(monkeypatch, cast, bias):
    head, codes, scale, b = _cpu_head(monkeypatch, bias)
    model = torch.nn.Sequential(torch.nn.Linear(4, 4), head)
    cast(model)
    assert head.codes.dtype == torch.float8_e4m3fn and head.scale.dtype == torch.float32
    assert torch.equal(head.codes.view(torch.uint8), codes.view(torch.uint8))
    assert torch.equal(head.scale, scale)
    assert (head.bias is None) if b is None else torch.equal(head.bias, b)
    # the rest of the model is cast as ever
    assert model[0].weight.dtype == cast(torch.nn.Linear(1, 1)).weight.dtype
    # and the state comes back as it went
    other, *_ = _cpu_head(monkeypatch, bias)
    other.codes.view(torch.uint8).zero_()
    other.scale.zero_()
    other.load_state_dict(head.state_dict())
    assert torch.equal(other.codes.view(torch.uint8), codes.view(torch.uint8))
    assert torch.equal(other.scale, scale)


def test_a_head_goes_to_another_device(monkeypatch):
    head, codes, *_ = _cpu_head(monkeypatch)
    head.to("meta", torch.bfloat16)
    assert head.codes.device.type == head.scale.device.type == head.bias.device.type == "meta"
    assert head.codes.dtype == torch.float8_e4m3fn and head.codes.shape == codes.shape
    head.to_empty(device="cpu")
    assert head.codes.device.type == "cpu" and head.codes.dtype == torch.float8_e4m3fn


def test_a_scorer_wants_one_target_per_row():
    """A longer target would score rows against their neighbours'."""
    from lm_head_projection_b200 import norm, scoring

    sc = scoring.Fp8Scorer(norm.AddRMSNorm(64), None)
    x = torch.zeros(2, 5, 64, dtype=torch.bfloat16)
    for shape in ((2, 6), (11,), (2, 4), (2,), (0,)):
        with pytest.raises(ValueError, match="target"):
            sc(x, None, torch.zeros(shape, dtype=torch.int64))
    for shape in ((2, 5), (10,), (2, 5, 1)):
        with pytest.raises(ValueError, match="CUDA"):
            sc(x, None, torch.zeros(shape, dtype=torch.int64))


def test_a_stream_of_another_device_is_refused():
    """Before anything is allocated or launched, by every call that takes one."""
    from types import SimpleNamespace

    from lm_head_projection_b200 import fp8, logprobs, norm

    st = SimpleNamespace(device=torch.device("cuda:1"))
    x, w = torch.zeros(4, 64), torch.ones(64)
    q, s1, s2 = torch.zeros(4, 64, dtype=torch.float8_e4m3fn), torch.ones(4, 1), torch.ones(1, 1)
    f = dict(stats=torch.zeros(4, 2), entropy=torch.zeros(4), top_ids=None)
    for call in (lambda: norm.add_rms_norm(x, w, stream=st),
                 lambda: norm.add_rms_norm_backward(x, x, w, stream=st),
                 lambda: norm.rms_norm_backward(x, x, w, stream=st),
                 lambda: norm.layer_norm_backward(x, x, w, stream=st),
                 lambda: fp8.quantize_rows(x, stream=st), lambda: fp8.quantize_blocks(x, stream=st),
                 lambda: fp8.block_matmul(q, s1, q, s2, stream=st),
                 lambda: logprobs.token_logprobs_forward(x, stream=st),
                 lambda: logprobs.token_logprobs_backward(x, None, f, stream=st)):
        with pytest.raises(ValueError, match="stream is of cuda:1"):
            call()
