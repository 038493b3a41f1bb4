"""What the scoring entry points refuse, on the host, without a GPU: the C ABI
returns before any launch and the Python layer raises before the call."""

from __future__ import annotations

import pytest
import torch

import lm_head_projection_b200 as pkg
from lm_head_projection_b200 import fp8, logprobs, norm, scoring

OK, INVALID, UNSUPPORTED = 0, 1, 2
no_gpu = pytest.mark.skipif(torch.cuda.is_available(),
                            reason="placeholder pointers must not reach a real device")
P = 4096  # placeholder, 16-byte aligned, never dereferenced
NAN = float("nan")


def _norm(X=P, res=0, W=P, rows=4, H=64, dtype=1, eps=1e-6, quant=0, Y=P, scale=0, Hs=0):
    return pkg.flkl_add_rms_norm_forward(X, res, W, rows, H, dtype, eps, quant, Y, scale, Hs, 0)


@no_gpu
@pytest.mark.parametrize("kw,want", [
    (dict(dtype=2), INVALID), (dict(rows=-1), INVALID), (dict(H=0), INVALID),
    (dict(eps=-1.0), INVALID), (dict(eps=NAN), INVALID), (dict(H=12), UNSUPPORTED),
    (dict(H=8200), UNSUPPORTED), (dict(rows=1 << 31), UNSUPPORTED), (dict(X=0), INVALID),
    (dict(W=0), INVALID), (dict(Y=0), INVALID), (dict(quant=1), INVALID),
    (dict(scale=P), INVALID), (dict(res=P), INVALID), (dict(Hs=P), INVALID),
    (dict(X=P + 8), UNSUPPORTED), (dict(quant=1, scale=P + 2), UNSUPPORTED),
    (dict(rows=0, X=0, Y=0), OK)])
def test_norm_forward_refusals(kw, want):
    assert _norm(**kw) == want


@no_gpu
def test_norm_backward_refusals():
    f = pkg.flkl_add_rms_norm_backward
    assert f(P, P, P, P, 4, 12, 1, 1e-6, 0, 1, P, 0, 0, 0, 0) == UNSUPPORTED
    assert f(P, P + 4, P, P, 4, 64, 1, 1e-6, 0, 1, P, 0, 0, 0, 0) == UNSUPPORTED
    assert f(P, P, P, P, 4, 64, 1, 1e-6, 1, 1, P, 0, 0, 0, 0) == INVALID
    assert f(P, P, P, P, 4, 64, 1, 1e-6, 1, 1, P, P, 0, 0, 0) == 5


@no_gpu
@pytest.mark.parametrize("kw,want", [
    (dict(dtype=2), INVALID), (dict(block=64), INVALID), (dict(cols=24), UNSUPPORTED),
    (dict(rows=-1), INVALID), (dict(cols=0), INVALID), (dict(src=0), INVALID),
    (dict(src=P + 8), UNSUPPORTED), (dict(q=P + 8), UNSUPPORTED), (dict(rows=0, src=0), OK)])
def test_quantize_refusals(kw, want):
    a = dict(src=P, rows=4, cols=64, dtype=1, block=1, q=P)
    a.update(kw)
    assert pkg.flkl_fp8_quantize(a["src"], a["rows"], a["cols"], a["dtype"], a["block"], a["q"],
                                 P, 0) == want


@no_gpu
@pytest.mark.parametrize("kw,want", [
    (dict(out=2), INVALID), (dict(M=-1), INVALID), (dict(N=-1), INVALID), (dict(K=0), INVALID),
    (dict(K=24), UNSUPPORTED), (dict(M=(1 << 30) + 1), UNSUPPORTED), (dict(A=0), INVALID),
    (dict(B=0), INVALID), (dict(sa=0), INVALID), (dict(sb=0), INVALID), (dict(D=0), INVALID),
    (dict(A=P + 8), UNSUPPORTED), (dict(B=P + 8), UNSUPPORTED), (dict(D=P + 1), UNSUPPORTED),
    (dict(sa=P + 2), UNSUPPORTED), (dict(bias=P + 1), UNSUPPORTED), (dict(M=0, A=0), OK),
    (dict(N=0, B=0), OK)])
def test_matmul_refusals(kw, want):
    a = dict(A=P, sa=P, B=P, sb=P, bias=0, M=4, N=8, K=64, out=1, D=P)
    a.update(kw)
    assert pkg.flkl_fp8_block_matmul(a["A"], a["sa"], a["B"], a["sb"], a["bias"], a["M"], a["N"],
                                     a["K"], a["out"], a["D"], 0) == want


_LP = dict(z=P, ld=64, t=P, rows=4, V=64, dtype=1, T=1.0, k=0, logp=P, ent=P, lse=P, stats=P,
           tl=0, ti=0)


@no_gpu
@pytest.mark.parametrize("kw,want", [
    (dict(dtype=2), INVALID), (dict(rows=-1), INVALID), (dict(V=0), INVALID),
    (dict(ld=63), INVALID), (dict(T=0.0), INVALID), (dict(T=NAN), INVALID),
    (dict(T=float("inf")), INVALID), (dict(T=1e-40), INVALID), (dict(k=-1), INVALID),
    (dict(k=33), UNSUPPORTED),
    (dict(V=8, k=9, tl=P, ti=P), UNSUPPORTED), (dict(k=4), INVALID), (dict(z=0), INVALID),
    (dict(t=0), INVALID), (dict(logp=0), INVALID), (dict(ent=0), INVALID),
    (dict(stats=P + 4), UNSUPPORTED), (dict(z=P + 1), UNSUPPORTED), (dict(t=P + 4), UNSUPPORTED),
    (dict(rows=0, z=0), OK)])
def test_logprobs_forward_refusals(kw, want):
    a = {**_LP, **kw}
    assert pkg.flkl_token_logprobs_forward(
        a["z"], a["ld"], a["t"], -100, a["rows"], a["V"], a["dtype"], a["T"], a["k"], a["logp"],
        a["ent"], a["lse"], a["stats"], a["tl"], a["ti"], 0) == want


@no_gpu
@pytest.mark.parametrize("kw,want", [
    (dict(dld=63), INVALID), (dict(z=0), INVALID), (dict(d=0), INVALID), (dict(stats=0), INVALID),
    (dict(t=0), INVALID), (dict(gt=P), INVALID), (dict(k=2, gt=P), INVALID),
    (dict(d=P + 1), UNSUPPORTED), (dict(T=-1.0), INVALID), (dict(rows=0, z=0), OK)])
def test_logprobs_backward_refusals(kw, want):
    a = dict(z=P, ld=64, t=P, rows=4, V=64, dtype=1, T=1.0, k=0, stats=P, ent=P, ti=0, gl=P, ge=P,
             gt=0, d=P, dld=64)
    a.update(kw)
    assert pkg.flkl_token_logprobs_backward(
        a["z"], a["ld"], a["t"], -100, a["rows"], a["V"], a["dtype"], a["T"], a["k"], a["stats"],
        a["ent"], a["ti"], a["gl"], a["ge"], a["gt"], a["d"], a["dld"], 0) == want


def test_python_layer_refusals():
    x, w = torch.zeros(4, 64, dtype=torch.bfloat16), torch.ones(64, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="CUDA"):
        norm.add_rms_norm(x, w)
    with pytest.raises(ValueError, match="dtype"):
        norm.add_rms_norm(x.half(), w.half())
    with pytest.raises(ValueError, match="residual"):
        norm.add_rms_norm(x, w, torch.zeros(4, 32, dtype=torch.bfloat16))
    with pytest.raises(ValueError, match="contiguous"):
        norm.add_rms_norm(torch.zeros(64, 4, dtype=torch.bfloat16).t(), w)
    with pytest.raises(ValueError, match="inplace"):
        norm.add_rms_norm(x, w, inplace=True)
    with pytest.raises(ValueError, match="dtype"):
        fp8.quantize_rows(x.half())
    with pytest.raises(ValueError, match="matrix"):
        fp8.quantize_blocks(torch.zeros(2, 4, 64))
    q = torch.zeros(4, 64, dtype=torch.float8_e4m3fn)
    s1, s2 = torch.ones(4, 1), torch.ones(1, 1)
    with pytest.raises(ValueError, match="CUDA"):
        fp8.block_matmul(q, s1, q, s2)
    with pytest.raises(ValueError, match="a_scale"):
        fp8.block_matmul(q, s2, q, s2)
    with pytest.raises(ValueError, match="b_scale"):
        fp8.block_matmul(q, s1, q, s1)
    with pytest.raises(ValueError, match="out_dtype"):
        fp8.block_matmul(q, s1, q, s2, out_dtype=torch.float16)
    with pytest.raises(ValueError, match="bias"):
        fp8.block_matmul(q, s1, q, s2, bias=torch.zeros(4))
    with pytest.raises(ValueError, match="out"):
        fp8.block_matmul(q, s1, q, s2, out=torch.zeros(4, 5, dtype=torch.bfloat16))
    z, t = torch.zeros(4, 64), torch.zeros(4, dtype=torch.int64)
    with pytest.raises(ValueError, match="CUDA"):
        logprobs.token_logprobs_forward(z, t)
    for k in (-1, 33):
        with pytest.raises(ValueError, match="top_k"):
            logprobs.token_logprobs_forward(z, t, top_k=k)
    with pytest.raises(ValueError, match="top_k"):
        logprobs.token_logprobs_forward(z[:, :8], t, top_k=9)
    with pytest.raises(ValueError, match="stride"):
        logprobs.token_logprobs_forward(z.t(), None)
    with pytest.raises(ValueError, match="stride"):
        logprobs.token_logprobs_forward(z[:1].expand(4, 64), t)
    with pytest.raises(ValueError, match="target"):
        logprobs.token_logprobs_forward(z, t.int())
    f = dict(stats=torch.zeros(4, 2), entropy=torch.zeros(4), top_ids=None)
    with pytest.raises(ValueError, match="target"):
        logprobs.token_logprobs_backward(z, None, f, dlogp=torch.zeros(4))
    with pytest.raises(ValueError, match="top_k"):
        logprobs.token_logprobs_backward(z, t, f, dtop_logp=torch.zeros(4, 2))
    with pytest.raises(ValueError, match="block_rows"):
        scoring.Fp8Scorer(norm.AddRMSNorm(64), None, block_rows=0)
