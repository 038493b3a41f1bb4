"""The scoring path on the GPU against the fp64 oracle: RMSNorm with the
residual's addition, e4m3 quantisers and products, token log-probabilities.

Tolerances, from the arithmetic (u = 2^-24, half a step of fp32):

* a result in bf16 is off by at most 2^-8 of itself, an e4m3 code by 2^-4 of
  the value or half the smallest step, 2^-10 of the scale;
* the norm: a sum of squares goes through at most 16 additions of a thread, 5
  of its warp and 16 of the CTA (37 u of a sum of positive terms, halved by the
  root), the reciprocal root (2 steps), and 4 products or quotients: below 32 u;
* a product's sums: at most K + K / 128 + 8 roundings, each of a step (2 u, the
  tensor cores may cut) of the sum of magnitudes;
* the softmax sums: a thread adds V / 128 terms (rows of 128 threads), then 20
  sums of sums, and a term 2^t has t (|t| < 32 where the term counts) off by 3
  roundings: S is off by at most (V / 128 + 20 + 3 * 32 + 4) u of itself, called
  tol(V).
"""

from __future__ import annotations

import numpy as np
import pytest
import torch

from oracle import scoring_oracle as o

pytestmark = pytest.mark.gpu
U = 2.0 ** -24
HALF = {"fp32": 2.0 ** -24, "bf16": 2.0 ** -8}
DT = {"fp32": torch.float32, "bf16": torch.bfloat16}


def _np(t):
    return None if t is None else t.detach().double().cpu().numpy()


def _close(got, want, bound, what=""):
    got, want, bound = np.asarray(got), np.asarray(want), np.asarray(bound)
    fin = np.isfinite(want)
    assert np.array_equal(np.isnan(got), np.isnan(want)), what
    assert np.array_equal(got[~fin & ~np.isnan(want)], want[~fin & ~np.isnan(want)]), what
    err = np.abs(got - np.where(fin, want, 0))[fin]
    b = np.broadcast_to(bound, want.shape)[fin]
    if err.size:
        i = np.argmax(err - b)
        assert (err <= b).all(), (what, err[i], b[i], want[fin][i])


# ------------------------------------------------------------------- norm
NORM_SIZES = [(1, 8), (5, 72), (33, 256), (7, 264), (3, 1024), (9, 1032), (130, 2056), (2, 4096),
              (3, 4104), (4, 8192)]


def _norm_inputs(rows, H, dtype, seed=0):
    g = torch.Generator().manual_seed(seed + rows * 7 + H)
    x, r = (torch.randn(rows, H, generator=g) * s for s in (1.0, 3.0))
    w = 1 + 0.1 * torch.randn(H, generator=g)
    return [t.to(DT[dtype]) for t in (x, r, w)]


@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
@pytest.mark.parametrize("rows,H", NORM_SIZES)
@pytest.mark.parametrize("residual", [True, False])
def test_norm_forward(dtype, rows, H, residual):
    from lm_head_projection_b200 import norm

    x, r, w = _norm_inputs(rows, H, dtype)
    xc, wc, rc = x.cuda(), w.cuda(), r.cuda() if residual else None
    got = norm.add_rms_norm(xc, wc, rc)
    q = norm.add_rms_norm(xc, wc, rc, quantize=True)
    y, h = o.add_rms_norm(_np(x), _np(r) if residual else None, _np(w), 1e-6, dtype)
    assert np.array_equal(_np(got["H"]), h) and np.array_equal(_np(q["H"]), h)
    assert (got["H"] is xc) == (not residual) and got["scale"] is None
    _close(_np(got["Y"]), y, np.abs(y) * (HALF[dtype] + 33 * U), "y")
    s = o.block_scales(y, 1)
    assert q["Y"].dtype == torch.float8_e4m3fn and q["scale"].shape == (rows, -(-H // 128))
    _close(_np(q["scale"]), s, s * 34 * U, "scale")
    sp = o.spread(_np(q["scale"]), rows, H, 1)
    _close(_np(q["Y"].float()) * sp, y, np.abs(y) * (2.0 ** -4 + 40 * U) + sp * 2.0 ** -10, "codes")


def test_norm_leading_dimensions_inplace_and_no_rows():
    from lm_head_projection_b200 import norm

    x, r, w = [t.cuda() for t in _norm_inputs(12, 256, "bf16")]
    want = norm.add_rms_norm(x, w, r, quantize=True)
    r2 = r.clone().view(3, 4, 256)
    got = norm.add_rms_norm(x.view(3, 4, 256), w, r2, quantize=True, inplace=True)
    assert got["Y"].shape == (3, 4, 256) and got["scale"].shape == (3, 4, 2)
    assert got["H"].data_ptr() == r2.data_ptr()
    for k in ("Y", "scale", "H"):
        assert torch.equal(got[k].flatten().float(), want[k].flatten().float()), k
    e = norm.add_rms_norm(x[:0], w, r[:0], quantize=True)
    assert e["Y"].shape == (0, 256) and e["scale"].shape == (0, 2)


def test_norm_of_zero_huge_and_non_finite_rows():
    from lm_head_projection_b200 import norm

    x = torch.randn(5, 384).cuda()
    x[0] = 0                      # codes 0, scale 1
    x[1, 128:256] = 0             # one block of zeros
    x[2, 3] = float("nan")        # the whole row
    x[3] *= 1e15                  # squares beyond fp32's comfort
    x[4, 5] = float("inf")
    w = torch.ones(384).cuda()
    q = norm.add_rms_norm(x, w, quantize=True)
    codes, s = q["Y"].float(), q["scale"]
    assert (codes[0] == 0).all() and (s[0] == 1).all()
    assert (codes[1, 128:256] == 0).all() and s[1, 1] == 1
    assert torch.isnan(codes[2]).all()
    y, _ = o.add_rms_norm(_np(x[3:4]), None, _np(w), 1e-6, "fp32")
    sp = o.spread(_np(s[3:4]), 1, 384, 1)
    _close(_np(codes[3:4]) * sp, y, np.abs(y) * (2.0 ** -4 + 40 * U) + sp * 2.0 ** -10)
    assert torch.isnan(codes[4, 5])  # infinity over infinity


@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
@pytest.mark.parametrize("rows,H", [(1, 8), (37, 200), (300, 2056), (70, 4104), (65, 8192)])
@pytest.mark.parametrize("cw,with_dh", [(True, True), (False, True), (True, False)])
def test_norm_backward(dtype, rows, H, cw, with_dh):
    from lm_head_projection_b200 import norm

    h, dy, w = _norm_inputs(rows, H, dtype, 3)
    dh = _norm_inputs(rows, H, dtype, 4)[0] if with_dh else None
    got = norm.add_rms_norm_backward(dy.cuda(), h.cuda(), w.cuda(),
                                     None if dh is None else dh.cuda(), compute_dW=cw)
    dx, dw = o.add_rms_norm_backward(_np(dy), _np(dh), _np(h), _np(w), 1e-6)
    # dx = dh + g / r - h c: each of the terms is off by at most 64 u of itself,
    # c's sum by 64 u of the sum of its magnitudes
    hh, g = _np(h), _np(dy) * _np(w)
    r = np.sqrt((hh * hh).mean(-1, keepdims=True) + 1e-6)
    mag = (np.abs(g) / r + np.abs(hh) * (np.abs(g * hh)).mean(-1, keepdims=True) / r ** 3
           + (0 if dh is None else np.abs(_np(dh))))
    _close(_np(got["dX"]), dx, np.abs(dx) * HALF[dtype] + mag * 128 * U, "dX")
    if cw:
        _close(_np(got["dW"]), dw, np.abs(_np(dy) * hh / r).sum(0) * (rows + 64) * U, "dW")
    else:
        assert got["dW"] is None
    if dh is None:  # the existing entry point's bits
        old = norm.rms_norm_backward(dy.cuda(), h.cuda(), w.cuda(), compute_dW=cw)
        assert torch.equal(old["dX"], got["dX"])


def test_add_rms_norm_module_gradients():
    from lm_head_projection_b200.norm import AddRMSNorm

    m = AddRMSNorm(136, dtype=torch.float32, device="cuda")
    x, r, w = [t.cuda() for t in _norm_inputs(6, 136, "fp32", 5)]
    with torch.no_grad():
        m.weight.copy_(w)
    x.requires_grad_(), r.requires_grad_()
    a, b = torch.randn(6, 136).cuda(), torch.randn(6, 136).cuda()
    y, h = m(x, r)
    ((y * a).sum() + (h * b).sum()).backward()
    dx, dw = o.add_rms_norm_backward(_np(a), _np(b), _np(x + r), _np(w), 1e-6)
    _close(_np(x.grad), dx, 1e-4 * np.abs(dx).max())
    assert torch.equal(x.grad, r.grad)
    _close(_np(m.weight.grad), dw, 1e-4 * np.abs(dw).max())
    # only h is used, only y is used, a frozen weight
    m.weight.requires_grad_(False)
    x.grad = r.grad = m.weight.grad = None
    m(x, r)[1].sum().backward()
    assert torch.equal(x.grad, torch.ones_like(x)) and m.weight.grad is None
    x.grad = None
    (m(x, r)[0] * a).sum().backward()
    dx, _ = o.add_rms_norm_backward(_np(a), None, _np(x + r), _np(w), 1e-6)
    _close(_np(x.grad), dx, 1e-4 * np.abs(dx).max())


# -------------------------------------------------------------- quantisers
@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
@pytest.mark.parametrize("rows,K", [(1, 16), (3, 112), (130, 128), (129, 144), (257, 1552), (5, 8192)])
@pytest.mark.parametrize("block", [1, 128])
def test_quantizers(dtype, rows, K, block):
    from lm_head_projection_b200 import fp8

    x = torch.randn(rows, K, generator=torch.Generator().manual_seed(rows + K)).to(DT[dtype])
    x[0, :16] = 0
    q, s = (fp8.quantize_rows if block == 1 else fp8.quantize_blocks)(x.cuda())
    xs = _np(x)
    want = o.block_scales(xs, block)
    _close(_np(s), want, want * U, "scale")  # one division
    sp = o.spread(_np(s), rows, K, block)
    _close(_np(q.float()) * sp, xs, np.abs(xs) * (2.0 ** -4 + 4 * U) + sp * 2.0 ** -10, "codes")
    # the block's extreme keeps its value
    assert (_np(q.float().abs().max())) == 448 or K == 16


# ----------------------------------------------------------------- product
def _product(M, N, K, out, bias, seed=0):
    from lm_head_projection_b200 import fp8

    g = torch.Generator().manual_seed(seed + M + 3 * N + 5 * K)
    a = torch.randn(M, K, generator=g) * torch.exp(torch.randn(M, 1, generator=g))
    b = torch.randn(N, K, generator=g) * 0.05
    bv = torch.randn(N, generator=g).to(DT[out]).cuda() if bias else None
    qa, sa = fp8.quantize_rows(a.cuda())
    qb, sb = fp8.quantize_blocks(b.cuda())
    got = fp8.block_matmul(qa, sa, qb, sb, bias=bv, out_dtype=DT[out])
    want, mag = o.block_matmul(_np(qa.float()), _np(sa), _np(qb.float()), _np(sb), _np(bv))
    _close(_np(got), want, np.abs(want) * HALF[out] + mag * 2 * (K + K // 128 + 8) * U)
    return qa, sa, qb, sb, got


@pytest.mark.parametrize("out,bias", [("bf16", False), ("fp32", True)])
@pytest.mark.parametrize("M,N,K", [
    (1, 1, 16), (1, 130, 128), (2, 1000, 144), (7, 129, 512), (16, 256, 256), (17, 384, 1552),
    (31, 127, 272), (33, 520, 4096), (64, 640, 384), (65, 1001, 640), (96, 300, 2064),
    (127, 128, 128), (128, 129, 1024), (129, 257, 256), (200, 1000, 1040), (256, 512, 512),
    (257, 513, 528), (300, 2050, 768), (640, 900, 1552)])
def test_block_matmul(M, N, K, out, bias):
    _product(M, N, K, out, bias)


@pytest.mark.parametrize("M", [1, 40, 300])
def test_block_matmul_wide_and_deep(M):
    _product(M, 20000, 512, "bf16", True)
    _product(M, 300, 14336, "fp32", False)


def test_block_matmul_empty_out_and_non_finite():
    from lm_head_projection_b200 import fp8

    qa, sa, qb, sb, d = _product(5, 200, 256, "bf16", False)
    assert fp8.block_matmul(qa[:0], sa[:0], qb, sb).shape == (0, 200)
    assert fp8.block_matmul(qa, sa, qb[:0], sb[:0]).shape == (5, 0)
    buf = torch.full((7, 200), 3.0, dtype=torch.bfloat16, device="cuda")
    r = fp8.block_matmul(qa, sa, qb, sb, out=buf[1:6])
    assert r.data_ptr() == buf[1:6].data_ptr() and torch.equal(buf[1:6], d)
    assert (buf[0] == 3).all() and (buf[6] == 3).all()
    # a NaN code or scale reaches its own row (or column) only
    q2 = qa.clone()
    q2.view(torch.uint8)[2, 200] = 0x7F
    s2 = sa.clone()
    s2[3, 0] = float("inf")
    got = fp8.block_matmul(q2, s2, qb, sb)
    assert torch.isnan(got[2]).all() and not torch.isfinite(got[3]).any()
    assert torch.equal(got[[0, 1, 4]], d[[0, 1, 4]])


@pytest.mark.parametrize("out", ["bf16", "fp32"])
@pytest.mark.parametrize("N", [1, 5, 64, 131, 250, 264])
def test_block_matmul_output_at_any_place(out, N):
    """D that starts anywhere in a 16-byte unit, rows of any phase: the outputs
    are the same and nothing beside them is touched."""
    from lm_head_projection_b200 import fp8

    for M in (129, 300):
        qa, sa, qb, sb, want = _product(M, N, 272, out, True)
        _, _, _, _, plain = _product(M, N, 272, out, False)
        for off in (0, 1, 3, 7):
            buf = torch.full((M * N + 24,), 7.0, dtype=DT[out], device="cuda")
            d = buf[off:off + M * N].view(M, N)
            fp8.block_matmul(qa, sa, qb, sb, out_dtype=DT[out], out=d)
            assert torch.equal(d, plain)
            assert (buf[:off] == 7).all() and (buf[off + M * N:] == 7).all()


@pytest.mark.parametrize("out", ["bf16", "fp32"])
@pytest.mark.parametrize("M,N,K", [
    (300, 2600, 272), (300, 2601, 1040), (257, 4607, 16), (512, 4352, 656),   # 128-wide tiles
    (520, 3303, 272), (1000, 2504, 1040), (300, 5001, 144), (769, 2900, 16)])  # 256-wide
def test_block_matmul_of_cta_pairs(M, N, K, out):
    """Both tile widths of the pairs: rows of any phase, ends inside tiles, several
    tiles a pair, a bias; nothing beside D is touched."""
    from lm_head_projection_b200 import fp8

    qa, sa, qb, sb, want = _product(M, N, K, out, False)
    _product(M, N, K, out, True)
    for off in (0, 3):
        buf = torch.full((M * N + 24,), 7.0, dtype=DT[out], device="cuda")
        d = buf[off:off + M * N].view(M, N)
        fp8.block_matmul(qa, sa, qb, sb, out_dtype=DT[out], out=d)
        assert torch.equal(d, want)
        assert (buf[:off] == 7).all() and (buf[off + M * N:] == 7).all()


@pytest.mark.parametrize("out", ["bf16", "fp32"])
@pytest.mark.parametrize("M,N,K", [(3400, 1, 272), (3600, 8, 144), (4100, 40, 16), (3333, 67, 144)])
def test_block_matmul_of_many_rows_and_few_columns(M, N, K, out):
    """Outputs narrower than a tile, a box and a 16-byte unit."""
    _product(M, N, K, out, False)
    _product(M, N, K, out, True)


def test_block_matmul_too_deep_for_the_small_kernel():
    """So deep that the tokens' scales leave no room for its ring: sampled columns
    against fp64."""
    from lm_head_projection_b200 import fp8

    M, N, K = 3, 9601, 67216
    g = torch.Generator(device="cuda").manual_seed(5)
    r = lambda *s: torch.randn(*s, device="cuda", generator=g)
    qa, sa = fp8.quantize_rows(r(M, K))
    qb = torch.empty(N, K, dtype=torch.float8_e4m3fn, device="cuda")
    sb = torch.empty(-(-N // 128), -(-K // 128), device="cuda")
    for i in range(0, N, 1280):  # whole blocks of rows at a time
        qb[i:i + 1280], sb[i // 128:i // 128 + 10] = fp8.quantize_blocks(r(min(1280, N - i), K))
    d = fp8.block_matmul(qa, sa, qb, sb, out_dtype=torch.float32)
    cols = [0, 127, 128, 4999, 9599, 9600]
    b = _np(qb[cols].float()) * np.repeat(_np(sb)[np.array(cols) // 128], 128, 1)[:, :K]
    a = _np(qa.float()) * np.repeat(_np(sa), 128, 1)[:, :K]
    _close(_np(d[:, cols]), a @ b.T, (np.abs(a) @ np.abs(b).T) * 2 * (K + K // 128 + 8) * U)


@pytest.mark.parametrize("M", [3, 130])
def test_block_matmul_rows_do_not_depend_on_the_batch(M):
    """Twice the same, and (within one kernel's range of M) a row's result does
    not depend on the rows beside it."""
    from lm_head_projection_b200 import fp8

    qa, sa, qb, sb, d = _product(M, 1000, 1040, "fp32", False)
    assert torch.equal(fp8.block_matmul(qa, sa, qb, sb, out_dtype=torch.float32), d)
    perm = torch.randperm(M, device="cuda")
    got = fp8.block_matmul(qa.view(torch.uint8)[perm].view(torch.float8_e4m3fn).contiguous(),
                           sa[perm].contiguous(), qb, sb, out_dtype=torch.float32)
    assert torch.equal(got, d[perm])


def test_block_matmul_output_past_32_bits():
    """M * N above 2^31: the last rows and columns, against fp64."""
    from lm_head_projection_b200 import fp8

    M, N, K = 17000, 131072, 128
    g = torch.Generator(device="cuda").manual_seed(1)
    qa, sa = fp8.quantize_rows(torch.randn(M, K, device="cuda", generator=g))
    qb, sb = fp8.quantize_blocks(torch.randn(N, K, device="cuda", generator=g))
    d = fp8.block_matmul(qa, sa, qb, sb)
    rows = [0, 1, 8191, 16384, 16385, M - 130, M - 1]
    want, mag = o.block_matmul(_np(qa.float()[rows]), _np(sa[rows]), _np(qb.float()), _np(sb))
    _close(_np(d[rows]), want, np.abs(want) * HALF["bf16"] + mag * 2 * (K + 9) * U)


def test_fp8_head_module():
    from lm_head_projection_b200 import fp8

    w = (torch.randn(1000, 256) * 0.05).bfloat16().cuda()
    x = torch.randn(2, 9, 256).bfloat16().cuda()
    b = torch.randn(1000).bfloat16().cuda()
    head = fp8.Fp8Head(w, b, out_dtype=torch.float32)
    z = head(x)
    assert z.shape == (2, 9, 1000) and z.dtype == torch.float32
    q, s = fp8.quantize_rows(x)
    want, mag = o.block_matmul(_np(q.float()).reshape(18, 256), _np(s).reshape(18, 2),
                               _np(head.codes.float()), _np(head.scale), _np(b))
    _close(_np(z).reshape(18, 1000), want, np.abs(want) * U + mag * 2 * 266 * U)


# ---------------------------------------------------------- log-probabilities
def tol(V):
    return (V / 128 + 20 + 96 + 4) * U


def _check_logprobs(z, t, k=0, T=1.0, grads=True, seed=0):
    """z on the GPU ([rows, V], any stride); compares everything."""
    from lm_head_projection_b200 import logprobs

    rows, V = z.shape
    dt = "bf16" if z.dtype == torch.bfloat16 else "fp32"
    got = logprobs.token_logprobs_forward(z, t, temperature=T, top_k=k)
    zn, tn = _np(z), None if t is None else t.cpu().numpy()
    want = o.token_logprobs(zn, tn, -100, T, k)
    # logp: (z - m) / T off by 2 roundings, ln S by tol(V) and a rounding
    b = lambda v: np.abs(np.where(np.isfinite(v), v, 0)) * 8 * U + 2 * tol(V)
    if t is not None:
        _close(_np(got["logp"]), want["logp"], b(want["logp"]), "logp")
    else:
        assert got["logp"] is None
    lse32 = np.abs(np.where(np.isfinite(want["lse"]), want["lse"], 0)) * 4 * U + 2 * tol(V)
    _close(_np(got["lse"]), want["lse"], lse32, "lse")
    # entropy = ln S - A / S, A's terms have the magnitude of the entropy and ln S
    ent = np.where(np.isfinite(want["entropy"]), want["entropy"], 0)
    _close(_np(got["entropy"]), want["entropy"], (3 + 2 * ent + 2 * np.log(V)) * tol(V), "entropy")
    if k:
        assert np.array_equal(got["top_ids"].cpu().numpy(), want["top_ids"])
        _close(_np(got["top_logp"]), want["top_logp"], b(want["top_logp"]), "top_logp")
    if not grads:
        return got
    rs = np.random.RandomState(seed)
    gl = rs.normal(size=rows).astype(np.float32) if t is not None else None
    ge = rs.normal(size=rows).astype(np.float32)
    gt = rs.normal(size=(rows, k)).astype(np.float32) if k else None
    c = lambda a: None if a is None else torch.from_numpy(a).cuda()
    for use in ((gl, ge, gt), (gl, None, None), (None, ge, None), (None, None, gt)):
        if use[0] is None and use[1] is None and use[2] is None:
            continue
        dz = logprobs.token_logprobs_backward(z, t, got, c(use[0]), c(use[1]), c(use[2]),
                                              temperature=T)
        assert dz.shape == z.shape and dz.dtype == z.dtype
        wz, mag = o.token_logprobs_backward(zn, tn, want, *use, -100, T)
        # p off by tol(V) and its exponent's roundings (|ln p| < 100 where p is
        # not 0 in fp32: 8 u of 145), the rest a few roundings
        _close(_np(dz), wz, np.abs(wz) * HALF[dt] + mag * (4 * tol(V) + 1200 * U)
               + 2.0 ** -126 * 1e3, "dz")
    return got


def _logits(rows, V, dtype, seed=0, pad=0, off=0):
    g = torch.Generator().manual_seed(seed * 1000 + rows + V)
    z = torch.randn(rows, V + pad + off, generator=g) * 3
    t = torch.randint(0, V, (rows,), generator=g)
    return z.to(DT[dtype]).cuda()[:, off:off + V], t.cuda()


@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
@pytest.mark.parametrize("rows,V,k", [
    (1, 1, 1), (2, 2, 2), (3, 7, 0), (2, 31, 31), (5, 33, 32), (1, 255, 5), (4, 1000, 20),
    (2, 2047, 1), (3, 2056, 32), (2, 8192, 8), (3, 8200, 20), (1, 50257, 32), (2, 128256, 20),
    (300, 500, 3), (1, 151936, 1)])
def test_logprobs(dtype, rows, V, k):
    z, t = _logits(rows, V, dtype)
    _check_logprobs(z, t, k, T=0.7 if V % 2 else 1.0)


@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
@pytest.mark.parametrize("pad,off", [(1, 0), (7, 1), (0, 3), (5, 8), (64, 5)])
def test_logprobs_padded_and_unaligned_rows(dtype, pad, off):
    z, t = _logits(5, 4099, dtype, pad=pad, off=off)
    assert not z.is_contiguous()
    _check_logprobs(z, t, 20, T=1.3)


@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
@pytest.mark.parametrize("V", [5, 3000, 20001])
def test_logprobs_masks(dtype, V):
    """Half the row masked, all of it, all but one, with -infinity and with the
    type's lowest value."""
    for low in (-float("inf"), torch.finfo(DT[dtype]).min):
        z, t = _logits(6, V, dtype, 1)
        z = z.clone()
        z[0, ::2] = low
        z[1] = low
        z[2] = low
        z[2, V // 2] = 1.5
        z[3, : V - 1] = low
        t[0], t[1] = 0, 1
        for T in (1.0, 0.6):
            if T < 1 and low != -float("inf"):
                continue  # the row of lowest values: its lse leaves fp32
            _check_logprobs(z, t, min(V, 20), T=T)


@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
@pytest.mark.parametrize("scale", [1e-30, 1e-3, 3e4, 1e30, 3e37])
def test_logprobs_magnitudes(dtype, scale):
    """Logits and temperatures of any size, with masked places: what a maximum less
    200 powers of two is rounds to the maximum, or leaves the type's range."""
    z, t = _logits(5, 6007, dtype, 11)
    z = (z.float() * scale / 3).to(DT[dtype])
    z[0, ::3] = -float("inf")
    z[1, 1::2] = torch.finfo(DT[dtype]).min
    z[2] = z[2, 0]
    t[0], t[1] = 1, 0
    _check_logprobs(z, t, 7, T=float(np.float32(scale)), grads=scale < 1e20)
    if scale == 3e4:  # differences far beyond what an exponential holds
        _check_logprobs(z, t, 7, T=1.0)


@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
@pytest.mark.parametrize("V", [40, 9000, 33000])
def test_logprobs_orders_that_fill_the_list(dtype, V):
    """Equal logits, ascending and descending rows, blocks of ties, zeros of
    both signs."""
    z = torch.zeros(7, V)
    a = torch.arange(V).float() / V * 8
    z[1] = a
    z[2] = -a
    z[3] = (torch.arange(V) // 7 % 5).float()
    z[4, ::3] = -0.0
    z[5] = a
    z[5, V // 2:] = 4.0
    z[6, V - 1] = 1.0
    t = torch.arange(7) % V
    _check_logprobs(z.to(DT[dtype]).cuda(), t.cuda(), 32)
    _check_logprobs(z.to(DT[dtype]).cuda(), t.cuda(), 1)


@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
@pytest.mark.parametrize("rows", [1, 37, 74, 75, 149, 297])
def test_logprobs_rows_split_over_clusters(dtype, rows):
    """8, 4, 2 and 1 CTAs per row: random rows, ties across the parts' borders,
    largest logits at the row's ends."""
    V = 33003
    z, t = _logits(rows, V, dtype, 9)
    z = z.clone()
    z[0, ::4000] = 20.0
    z[-1, -1] = 30.0
    z[-1, 0] = 30.0
    z[rows // 2, 5:] = 1.0
    _check_logprobs(z, t, 20, grads=rows == 37)


@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
@pytest.mark.parametrize("rows,V", [(2, 20003), (300, 20003), (300, 90001)])
def test_logprobs_few_tokens_left_by_a_mask(dtype, rows, V):
    """Fewer tokens left than alternatives asked for: the masked ones follow in
    index order."""
    for low in (-float("inf"), torch.finfo(DT[dtype]).min):
        z = torch.full((rows, V), low)
        z[:, V - 2] = 2.0
        z[:, 19000] = 2.0
        z[:, 77] = -1.0
        z[0, 77] = low
        t = torch.full((rows,), 77)
        _check_logprobs(z.to(DT[dtype]).cuda(), t.cuda(), 20, grads=rows == 2)
        _check_logprobs(z.to(DT[dtype]).cuda(), t.cuda(), 1, grads=False)


@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
@pytest.mark.parametrize("V", [40000, 128256])
def test_logprobs_large_logits_of_few_threads(dtype, V):
    """What passes the bound sits in few threads' parts and overflows the list."""
    rows = 300
    e = 4 if dtype == "fp32" else 8
    z, t = _logits(rows, V, dtype, 10)
    v = torch.arange(V, device="cuda") // e % 256
    z[:, v < 20] += 40.0
    z[1, v < 20] = 33.0
    _check_logprobs(z, t, 32, grads=False)
    _check_logprobs(z, t, 2, grads=False)


@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
def test_logprobs_non_finite_rows(dtype):
    z, t = _logits(5, 5000, dtype, 2)
    z = z.clone()
    z[0, 77] = float("nan")
    z[0, 4000] = float("nan")
    z[1, 4999] = float("inf")
    z[2] = -float("inf")
    z[2, 9] = float("nan")
    z[3, 0] = -float("nan")
    got = _check_logprobs(z, t, 5, grads=False)
    assert list(got["top_ids"][0, :2].tolist()) == [77, 4000]


@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
def test_logprobs_dropped_and_foreign_targets(dtype):
    z, t = _logits(6, 3001, dtype, 3)
    t[0], t[1], t[2], t[3] = -100, 3001, -1, 1 << 40
    z = z.clone()
    z[0] = float("nan")  # a dropped row is not looked at
    got = _check_logprobs(z, t, 4)
    assert got["logp"][0] == 0 and (got["top_ids"][0] == -1).all()
    assert (got["logp"][1:4] == 0).all() and (got["entropy"][1:4] > 0).all()
    _check_logprobs(z[1:], None, 4)


def test_logprobs_target_among_the_alternatives_and_peaked_rows():
    z, _ = _logits(4, 6000, "fp32", 4)
    z = z.clone()
    t = z.argmax(1)
    z[1, t[1]] += 40.0  # p = 1 to the last bit
    z[2, t[2]] += 8.0
    _check_logprobs(z, t, 3)


def test_logprobs_no_rows_and_long_rows():
    from lm_head_projection_b200 import logprobs

    z = torch.empty(0, 100, device="cuda")
    r = logprobs.token_logprobs_forward(z, torch.empty(0, dtype=torch.int64, device="cuda"), top_k=3)
    assert r["logp"].shape == (0,) and r["top_ids"].shape == (0, 3)
    assert logprobs.token_logprobs_backward(z, None, r, dentropy=r["entropy"]).shape == (0, 100)
    z, t = _logits(2, 1000003, "bf16", 5)
    _check_logprobs(z, t, 8)


def test_logprobs_offsets_past_32_bits():
    """rows * stride above 2^31 elements: the last rows."""
    from lm_head_projection_b200 import logprobs

    rows, V = 16500, 131100
    z = torch.empty(rows, V, dtype=torch.bfloat16, device="cuda")
    z[:-3].fill_(0)
    tail, tt = _logits(3, V, "bf16", 6)
    z[-3:] = tail
    t = torch.full((rows,), -100, device="cuda")
    t[-3:] = tt
    got = logprobs.token_logprobs_forward(z, t, top_k=4)
    want = o.token_logprobs(_np(tail), tt.cpu().numpy(), -100, 1.0, 4)
    assert np.array_equal(got["top_ids"][-3:].cpu().numpy(), want["top_ids"])
    _close(_np(got["logp"][-3:]), want["logp"], np.abs(want["logp"]) * 8 * U + 2 * tol(V))
    gl = torch.ones(rows, device="cuda")
    dz = logprobs.token_logprobs_backward(z, t, got, dlogp=gl)
    wz, mag = o.token_logprobs_backward(_np(tail), tt.cpu().numpy(), want, np.ones(3))
    _close(_np(dz[-3:]), wz, np.abs(wz) * 2.0 ** -8 + mag * (4 * tol(V) + 1200 * U) + 1e-30)
    assert torch.count_nonzero(dz[:-3]) == 0


def test_token_logprobs_autograd():
    from lm_head_projection_b200.logprobs import TokenLogProbs, token_logprobs

    z, t = _logits(5, 700, "fp32", 7, pad=20)
    t[3] = -100
    buf = z.clone().requires_grad_()
    r = TokenLogProbs(temperature=0.8, top_k=6)(buf, t)
    g = torch.Generator().manual_seed(1)
    gl, ge, gt = (torch.randn(*s, generator=g).cuda() for s in ((5,), (5,), (5, 6)))
    ((r.logp * gl).sum() + (r.entropy * ge).sum() + (r.top_logp * gt).sum()).backward()
    want = o.token_logprobs(_np(z), t.cpu().numpy(), -100, 0.8, 6)
    wz, mag = o.token_logprobs_backward(_np(z), t.cpu().numpy(), want, _np(gl), _np(ge), _np(gt),
                                        -100, 0.8)
    _close(_np(buf.grad), wz, mag * (4 * tol(700) + 1200 * U))
    # against differences of the forward: one logit of each kept row
    buf.grad = None
    token_logprobs(buf, t, temperature=0.8).entropy.sum().backward()
    for c in (int(t[0]), 11):
        e = torch.zeros_like(z)
        e[0, c] = 0.05
        f = lambda v: float(token_logprobs(v, t, temperature=0.8).entropy.double().sum())
        num = (f(z + e) - f(z - e)) / 0.1
        assert abs(num - float(buf.grad[0, c])) < 2e-3 * max(1e-2, abs(num)) + 1e-4


def test_second_gradients_are_refused():
    from lm_head_projection_b200.logprobs import token_logprobs
    from lm_head_projection_b200.norm import AddRMSNorm

    z, t = _logits(3, 50, "fp32")
    z.requires_grad_()
    g, = torch.autograd.grad(token_logprobs(z, t).logp.pow(2).sum(), z, create_graph=True)
    with pytest.raises(RuntimeError, match="once_differentiable"):
        g.sum().backward()
    m = AddRMSNorm(64, dtype=torch.float32, device="cuda")
    x, r, _ = [v.cuda().requires_grad_() for v in _norm_inputs(3, 64, "fp32")]
    g, = torch.autograd.grad(m(x, r)[0].pow(2).sum(), x, create_graph=True)
    with pytest.raises(RuntimeError, match="once_differentiable"):
        g.sum().backward()


# ------------------------------------------------- streams, graphs, the chain
def _chain():
    from lm_head_projection_b200.fp8 import Fp8Head
    from lm_head_projection_b200.norm import AddRMSNorm
    from lm_head_projection_b200.scoring import Fp8Scorer

    torch.manual_seed(0)
    H, V = 512, 5000
    n = AddRMSNorm(H, device="cuda")
    head = Fp8Head((torch.randn(V, H) * 0.1).bfloat16().cuda(), out_dtype=torch.float32)
    x, r = (torch.randn(3, 50, H).bfloat16().cuda() for _ in range(2))
    t = torch.randint(0, V, (3, 50)).cuda()
    t[1, 40:] = -100
    return n, head, x, r, t, lambda **kw: Fp8Scorer(n, head, top_k=5, temperature=0.9, **kw)


@pytest.mark.parametrize("block_rows", [1024, 64, 7])
def test_the_operators_together(block_rows):
    """Norm, head and log-probabilities as a scorer runs them, against the fp64
    chain of the kernels' own codes (a code at a border may go either way)."""
    n, head, x, r, t, scorer = _chain()
    out = scorer(block_rows=block_rows)(x, r, t)
    q, s, h = n.quantized(x, r)
    assert torch.equal(out["H"], h) and out["logp"].shape == (3, 50)
    z, mag = o.block_matmul(_np(q.float()).reshape(150, -1), _np(s).reshape(150, -1),
                            _np(head.codes.float()), _np(head.scale))
    want = o.token_logprobs(z, t.reshape(-1).cpu().numpy(), -100, 0.9, 5)
    dz = (mag * 2 * (512 + 12) * U).max() + np.abs(z).max() * U  # logits off by this at most
    _close(_np(out["logp"]).reshape(-1), want["logp"], 2 * dz / 0.9 + 4 * tol(5000))
    _close(_np(out["top_logp"]).reshape(150, 5), want["top_logp"], 2 * dz / 0.9 + 4 * tol(5000))
    kept = (t.reshape(-1) != -100).cpu().numpy()
    ids = out["top_ids"].reshape(150, 5).cpu().numpy()
    got = np.take_along_axis(z, np.maximum(ids, 0), 1)
    ref = np.take_along_axis(z, np.maximum(want["top_ids"], 0), 1)
    assert (np.abs(got - ref)[kept] <= 2 * dz).all() and (ids[~kept] == -1).all()


@pytest.mark.parametrize("rows", [1, 40, 300])
def test_side_stream_and_captured_graph(rows):
    """The whole chain on another stream and replayed from a graph with new
    inputs gives the direct call's bits."""
    n, head, x, r, t, scorer = _chain()
    sc = scorer()
    x, r, t = x.reshape(150, -1).repeat(2, 1)[:rows].contiguous(), \
        r.reshape(150, -1).repeat(2, 1)[:rows].contiguous(), t.reshape(-1).repeat(2)[:rows].contiguous()
    want = sc(x, r, t)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        got = sc(x, r, t)
    side.synchronize()
    for k in want:
        assert torch.equal(got[k], want[k]), k
    graphs = []
    for _ in range(2):
        xs, rs, ts = x.clone(), r.clone(), t.clone()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            out = sc(xs, rs, ts)
        graphs.append((g, xs, rs, ts, out))
    x2 = torch.randn_like(x)
    graphs[0][1].copy_(x2)
    for g in (graphs[0][0], graphs[1][0], graphs[0][0]):
        g.replay()
    torch.cuda.synchronize()
    want2 = sc(x2, r, t)
    for k in want:
        assert torch.equal(graphs[1][4][k], want[k]), k
        assert torch.equal(graphs[0][4][k], want2[k]), k


def test_calls_with_a_stream_of_their_own():
    """Every call on the stream it is given, its allocations too, while the
    current stream is busy with other work."""
    from lm_head_projection_b200 import fp8, logprobs, norm

    x, r, w = [t.cuda() for t in _norm_inputs(40, 512, "bf16")]
    z, t = _logits(40, 3000, "bf16", 8)
    qb, sb = fp8.quantize_blocks(torch.randn(700, 512, device="cuda"))

    def chain(**kw):
        f = norm.add_rms_norm(x, w, r, quantize=True, **kw)
        b = norm.add_rms_norm_backward(x, f["H"], w, dH=r, **kw)
        q, s = fp8.quantize_rows(x, **kw)
        d = fp8.block_matmul(q, s, qb, sb, **kw)
        l = logprobs.token_logprobs_forward(z, t, top_k=4, **kw)
        g = logprobs.token_logprobs_backward(z, t, l, dentropy=l["entropy"], **kw)
        return [f["Y"].float(), f["scale"], f["H"], b["dX"], b["dW"], q.float(), d, l["logp"], g]

    want = chain()
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    got = []
    for _ in range(4):
        for _ in range(20):
            junk = torch.randn(64, 4096, device="cuda") * 2  # what the current stream reuses
        got.append(chain(stream=side))
        side.synchronize()
    torch.cuda.synchronize()
    for g in got:
        for a, b in zip(g, want):
            assert torch.equal(a, b)


def test_two_streams_at_once():
    n, head, x, r, t, scorer = _chain()
    sc = scorer()
    x2 = torch.randn_like(x)
    want = [sc(x, r, t), sc(x2, r, t)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    got = [[], []]
    for _ in range(5):
        for i, xi in enumerate((x, x2)):
            with torch.cuda.stream(streams[i]):
                got[i].append(sc(xi, r, t))
    torch.cuda.synchronize()
    for i in range(2):
        for o_ in got[i]:
            for k in want[i]:
                assert torch.equal(o_[k], want[i][k]), k


_FIRST_CALLS_IN_A_GRAPH = """
import sys; sys.path.insert(0, sys.argv[1])
import torch
from lm_head_projection_b200 import fp8, logprobs, norm
g = torch.Generator(device="cuda").manual_seed(0)
r = lambda *s: torch.randn(*s, device="cuda", generator=g)
x, h, w, wt, z = r(200, 512).bfloat16(), r(200, 512).bfloat16(), r(512).bfloat16(), r(1000, 512), r(6, 3000)
t = torch.randint(0, 3000, (6,), device="cuda", generator=g)
def step():
    f = norm.add_rms_norm(x, w, h, quantize=True)
    b = norm.add_rms_norm_backward(x, f["H"], w, dH=h)
    qb, sb = fp8.quantize_blocks(wt)
    d = fp8.block_matmul(f["Y"], f["scale"], qb, sb)
    e = fp8.block_matmul(f["Y"][:9], f["scale"][:9], qb, sb)
    l = logprobs.token_logprobs_forward(z, t, top_k=3)
    return [b["dX"], b["dW"], d, e, l["logp"], l["top_ids"],
            logprobs.token_logprobs_backward(z, t, l, dlogp=l["logp"])]
graph = torch.cuda.CUDAGraph()
with torch.cuda.graph(graph):
    out = step()
graph.replay()
torch.cuda.synchronize()
assert all(torch.equal(a, b) for a, b in zip(out, step()))
from lm_head_projection_b200 import flkl_fp8_device_status, flkl_norm_device_status
assert flkl_fp8_device_status() == 0 and flkl_norm_device_status() == 0
"""


def test_first_calls_of_a_process_inside_a_graph():
    """Nothing of a first call (attributes, driver entry points, occupancy) is
    forbidden while a stream is captured."""
    import subprocess
    import sys
    from pathlib import Path

    root = Path(__file__).resolve().parent.parent
    r = subprocess.run([sys.executable, "-c", _FIRST_CALLS_IN_A_GRAPH, str(root)],
                       capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stderr[-2000:]


def test_autograd_step_captured():
    """The modules' forward and backward in a graph, warmed up on a side stream."""
    from lm_head_projection_b200.logprobs import TokenLogProbs
    from lm_head_projection_b200.norm import AddRMSNorm

    m, lp = AddRMSNorm(256, device="cuda"), TokenLogProbs(top_k=3)
    x, r, w = [t.cuda() for t in _norm_inputs(30, 256, "bf16")]
    x.requires_grad_()
    t = torch.randint(0, 256, (30,)).cuda()

    def step():
        m.weight.grad = x.grad = None
        y, h = m(x, r)
        o_ = lp(y, t)
        (o_.logp.sum() + o_.entropy.sum() + o_.top_logp.sum() + h.float().sum()).backward()

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        for _ in range(3):
            step()
    torch.cuda.current_stream().wait_stream(side)
    want = [x.grad.clone(), m.weight.grad.clone()]
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step()
    got = [x.grad, m.weight.grad]
    for v in got:
        v.zero_()
    g.replay()
    torch.cuda.synchronize()
    for a, b in zip(got, want):
        assert torch.equal(a, b)


def test_training_step_captured_while_an_eager_one_lives():
    """Forward and backward of norm and log-probabilities inside a graph."""
    from lm_head_projection_b200 import logprobs, norm

    x, r, w = [t.cuda() for t in _norm_inputs(64, 512, "bf16")]
    z, t = _logits(64, 3000, "bf16", 8)
    z = z.contiguous()

    def step():
        f = norm.add_rms_norm(x, w, r)
        b = norm.add_rms_norm_backward(f["Y"], f["H"], w, dH=x)
        l = logprobs.token_logprobs_forward(z, t, top_k=4)
        d = logprobs.token_logprobs_backward(z, t, l, dlogp=l["logp"], dentropy=l["entropy"],
                                             dtop_logp=l["top_logp"])
        return [f["Y"], f["H"], b["dX"], b["dW"], l["logp"], l["top_ids"], d]

    eager = step()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out = step()
    for v in out:
        v.zero_()
    g.replay()
    torch.cuda.synchronize()
    for a, b in zip(eager, out):
        assert torch.equal(a, b)
