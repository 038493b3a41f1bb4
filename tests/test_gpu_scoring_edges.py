"""Edges of the scoring path on the GPU, beside tests/test_gpu_scoring.py: codes at
exact ties, log-probabilities where logits over temperature leave fp32, waits of
the product that run out."""

from __future__ import annotations

import numpy as np
import pytest
import torch

import lm_head_projection_b200 as pkg
from oracle import scoring_oracle as o
from tests.test_gpu_scoring import DT, HALF, U, _close, _np, tol

pytestmark = pytest.mark.gpu


def _same_codes(codes, v, block_rows=1):
    """Codes are 448 v / max |v| rounded exactly (v in fp64, exact)."""
    m = o.block_scales(v, block_rows) * 448  # (only for its blocks' shape)
    for i in range(m.shape[0]):
        for j in range(m.shape[1]):
            r, c = slice(i * block_rows, (i + 1) * block_rows), slice(128 * j, 128 * j + 128)
            top = np.abs(v[r, c]).max()
            want = o.e4m3_quotients(v[r, c], top)
            assert np.array_equal(codes[r, c], want), (i, j)


# --------------------------------------------------------- codes at exact ties
@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
@pytest.mark.parametrize("block", [1, 128])
def test_quantizer_codes_of_every_pair_of_short_values(dtype, block):
    """Every significand of bf16 against every largest value's, over all the
    exponents that have a code: the nearest code, ties to even."""
    from lm_head_projection_b200 import fp8

    sig = np.arange(128, 256) / 128.0
    per = np.concatenate([sig * 2.0 ** -e for e in range(0, 20)])  # 2560 values
    rows = []
    for m in sig:
        v = np.where(per <= m, per, 0.0)
        blocks = np.zeros((21, 128))
        blocks[:, 0] = m
        blocks[:, 1:].reshape(-1)[:] = 0
        flat = np.zeros(21 * 127)
        flat[:v.size] = v
        blocks[:, 1:] = flat.reshape(21, 127)
        rows.append(blocks)
    x = np.concatenate(rows)  # [2688, 128]: a row is one block
    x[1::2] *= -1.0
    x[::3] *= 2.0 ** 40
    x[1::3] *= 2.0 ** -40
    x[5, 0] = x[5, 0] * 2.0 ** 126  # the largest of the type's range
    if block == 128:
        # a row of 128 x 128 blocks: each has one of the rows above, spread out
        y = np.zeros((128, 128 * len(x)))
        for i, row in enumerate(x):
            y[np.arange(128), 128 * i + (np.arange(128) * 37 + i) % 128] = row
        x = y
    t = torch.from_numpy(x).to(DT[dtype])
    assert np.array_equal(_np(t), x)
    q, _ = (fp8.quantize_rows if block == 1 else fp8.quantize_blocks)(t.cuda())
    _same_codes(_np(q.float()), x, block)


@pytest.mark.parametrize("rows,H", [(300, 136), (64, 1024), (33, 2048), (40, 4096), (30, 8192)])
@pytest.mark.parametrize("residual", [True, False])
def test_norm_codes_are_the_nearest(rows, H, residual):
    """bf16 rows: the codes of W h over the block's largest, in exact arithmetic;
    of random rows about one in two thousand lies at a tie."""
    from lm_head_projection_b200 import norm

    g = torch.Generator().manual_seed(rows + H)
    x, r = (torch.randn(rows, H, generator=g).bfloat16() for _ in range(2))
    w = (1 + 0.1 * torch.randn(H, generator=g)).bfloat16()
    x[0] = (x[0] * 16).round() / 16  # short values: many ties
    x[1] = x[1] * 2.0 ** 50
    x[2] = x[2] * 2.0 ** -30
    r[0] = 0
    w[: H // 2] = 1.0
    got = norm.add_rms_norm(x.cuda(), w.cuda(), r.cuda() if residual else None, quantize=True)
    p = _np(got["H"]) * _np(w)
    s = _np(got["scale"])
    # (where a block of y is below 2^-100 its codes are 0: none here)
    assert (s > 2.0 ** -90).all()
    _same_codes(_np(got["Y"].float()), p)
    y, _ = o.add_rms_norm(_np(got["H"]), None, _np(w), 1e-6, "bf16")
    want = o.block_scales(y, 1)
    # the sum of squares 37 u, halved by the root, its reciprocal and three products
    assert (np.abs(s - want) <= want * 32 * U).all()


def test_norm_codes_of_extreme_rows():
    """Rows whose sum of squares leaves fp32, zeros, tiny rows: as before."""
    from lm_head_projection_b200 import norm

    x = torch.randn(6, 256).cuda()
    x[0] = 1e-45
    x[1] = 1e-36
    x[2] *= 1e25          # squares overflow: r = 0
    x[3] = 0
    x[4, 7] = float("inf")
    x[5, 200] = float("nan")
    w = torch.ones(256).cuda()
    q = norm.add_rms_norm(x, w, quantize=True)
    c, s = q["Y"].float(), q["scale"]
    assert (c[:4] == 0).all() and (s[:4] == 1).all()
    assert torch.isnan(c[4, 7]) and (c[4, :7] == 0).all() and (c[4, 8:] == 0).all()
    assert torch.isnan(c[5]).all()


# ------------------------------------- log-probabilities beyond fp32's |m| / T
@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
@pytest.mark.parametrize("V", [7, 1000, 8192, 5003])
@pytest.mark.parametrize("m,T", [(-1e38, 1e-3), (-1e36, 1e-5), (-1e37, 1e-4), (1e38, 1e-3),
                                 (1e5, 1e-36), (-3e38, 0.5),
                                 # differences of logits beyond fp32 that count
                                 (2.9e38, 1.5e36), (-2e38, 2.4e36), (3e38, 3e38), (1e30, 3e38),
                                 (3e38, 4.0)])
def test_logprobs_of_rows_far_beyond_the_temperature(dtype, V, m, T):
    """Rows of one value, as a mask of a large finite number leaves them, whole,
    partly masked with -infinity or with one token left: the entropy is ln of the
    number of tokens that share the maximum and no gradient is NaN."""
    from lm_head_projection_b200 import logprobs

    T = float(np.float32(T))
    z = torch.full((5, V), m)
    z[1, 3:] = -float("inf")
    z[2, 1::2] = torch.finfo(DT[dtype]).min
    z[3, V // 2] = m * (0.9 if m < 0 else 1.1)
    z[4, ::3] = m * (1.1 if m < 0 else 0.9)
    z = z.to(DT[dtype]).cuda()
    t = torch.tensor([0, 1, 2, V // 2, 1]).cuda()
    k = min(V, 6)
    got = logprobs.token_logprobs_forward(z, t, temperature=T, top_k=k)
    zn, tn = _np(z), t.cpu().numpy()
    want = o.token_logprobs(zn, tn, -100, T, k)
    big = np.finfo(np.float32).max
    for n in ("logp", "top_logp"):  # (what leaves fp32 is infinite there)
        w = np.where(np.abs(want[n]) > big, np.copysign(np.inf, want[n]), want[n])
        fin = np.where(np.isfinite(w), w, 0)
        _close(_np(got[n]), w, np.abs(fin) * 8 * U + 2 * tol(V), n)
    assert np.array_equal(got["top_ids"].cpu().numpy(), want["top_ids"])
    ent = want["entropy"]
    _close(_np(got["entropy"]), ent, (3 + 2 * ent + 2 * np.log(V + 1)) * tol(V), "entropy")
    rs = np.random.RandomState(V)
    gl, ge = (rs.normal(size=5).astype(np.float32) for _ in range(2))
    gt = rs.normal(size=(5, k)).astype(np.float32)
    c = lambda a: None if a is None else torch.from_numpy(a).cuda()
    for use in ((gl, ge, gt), (gl, None, None), (None, ge, None)):
        dz = logprobs.token_logprobs_backward(z, t, got, c(use[0]), c(use[1]), c(use[2]),
                                              temperature=T)
        wz, mag = o.token_logprobs_backward(zn, tn, want, *use, -100, T)
        # as in test_gpu_scoring.py; what 1 / T makes smaller than fp32's normal
        # numbers may be cut
        _close(_np(dz), wz, np.abs(wz) * HALF[dtype] + mag * (4 * tol(V) + 1200 * U)
               + 2.0 ** -126, "dz")


# ------------------------------------------------- waits of the product that run out
def _product_inputs(M, N, K, seed=0):
    from lm_head_projection_b200 import fp8

    g = torch.Generator(device="cuda").manual_seed(seed + M + 3 * N + 5 * K)
    qa, sa = fp8.quantize_rows(torch.randn(M, K, device="cuda", generator=g))
    qb = torch.empty(N, K, dtype=torch.float8_e4m3fn, device="cuda")
    sb = torch.empty(-(-N // 128), -(-K // 128), device="cuda")
    for i in range(0, N, 1280):  # whole blocks of rows at a time
        qb[i:i + 1280], sb[i // 128:i // 128 + 10] = fp8.quantize_blocks(
            torch.randn(min(1280, N - i), K, device="cuda", generator=g))
    return qa, sa, qb, sb


@pytest.mark.parametrize("role", [1, 2, 3])
@pytest.mark.parametrize("M,N,K,at", [
    (5, 1000, 2048, 0), (5, 1000, 2048, 1),          # small kernel, clusters that share K
    (40, 40000, 2048, 0), (40, 40000, 2048, 21),     # several tiles a CTA
    (300, 2600, 2048, 0), (300, 2600, 2048, 3), (300, 2600, 2048, 9),     # pairs, 128 wide
    (3000, 5004, 2048, 1), (3000, 5004, 2048, 6), (3000, 5004, 2048, 20)])  # 256 wide
def test_a_product_whose_waits_run_out(M, N, K, at, role):
    """One role stops: the others give up after their limit, the kernel ends in
    good time, says so once, and the next product is right."""
    from lm_head_projection_b200 import fp8

    qa, sa, qb, sb = _product_inputs(M, N, K)
    want = fp8.block_matmul(qa, sa, qb, sb)
    assert pkg.flkl_fp8_device_status() == 0
    d = torch.zeros_like(want)
    a, b = (torch.cuda.Event(enable_timing=True) for _ in range(2))
    st = torch.cuda.current_stream().cuda_stream
    a.record()
    assert pkg.flkl_fp8_wait_selftest(qa.data_ptr(), sa.data_ptr(), qb.data_ptr(), sb.data_ptr(),
                                      M, N, K, d.data_ptr(), role, at, 20, st) == 0
    b.record()
    status = pkg.flkl_fp8_device_status(st)
    if M <= 64 and role == 3:  # the small kernel has no odd CTAs
        assert status == 0 and torch.equal(d, want)
    else:
        assert status == 4  # FLKL_ERR_TIMEOUT
        # a wait, the others' (which begin by then), and the loads' landing
        assert 15 < a.elapsed_time(b) < 100
    assert pkg.flkl_fp8_device_status(st) == 0
    assert torch.equal(fp8.block_matmul(qa, sa, qb, sb), want)
    assert pkg.flkl_fp8_device_status(st) == 0


# ------------------------------------------------------ gradients of spread rows
@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
@pytest.mark.parametrize("V,between", [(3000, 64), (3001, 7), (2999, 1), (3000, 100)])
def test_logprobs_gradient_of_one_position_of_many(dtype, V, between):
    """``logits[:, -1]`` of a batch of sequences: the gradient takes rows times V,
    not the whole sequences' memory, and holds the dense rows' bits."""
    from lm_head_projection_b200 import logprobs

    g = torch.Generator().manual_seed(V)
    z = torch.randn(6, between, V, generator=g).to(DT[dtype]).cuda()
    last = z[:, -1]
    assert between == 1 or not last.is_contiguous()
    t = torch.randint(0, V, (6,), generator=g).cuda()
    gl, ge = torch.randn(6, generator=g).cuda(), torch.randn(6, generator=g).cuda()
    f = logprobs.token_logprobs_forward(last, t)
    d = logprobs.token_logprobs_backward(last, t, f, dlogp=gl, dentropy=ge)
    assert d.shape == last.shape and d.stride(1) == 1 and V <= d.stride(0) < V + 8
    assert d.untyped_storage().nbytes() <= 6 * (V + 8) * z.element_size()
    dense = last.contiguous()
    want = logprobs.token_logprobs_backward(dense, t, f, dlogp=gl, dentropy=ge)
    assert torch.equal(d, want)
    # through autograd, into the whole tensor
    z.requires_grad_()
    r = logprobs.token_logprobs(z[:, -1], t)
    ((r.logp * gl).sum() + (r.entropy * ge).sum()).backward()
    assert torch.equal(z.grad[:, -1], want)
    assert between == 1 or (z.grad[:, :-1] == 0).all()


# ------------------------------------------------------------ the scorer's logits
@pytest.mark.parametrize("head_dtype", ["fp32", "bf16"])
@pytest.mark.parametrize("bias", [None, "fp32", "bf16"])
def test_scorer_scores_from_unrounded_logits(head_dtype, bias):
    """Whatever type the head gives its logits in, the scorer's log-probabilities
    are those of the fp32 product of the kernels' own codes."""
    from lm_head_projection_b200.fp8 import Fp8Head
    from lm_head_projection_b200.norm import AddRMSNorm
    from lm_head_projection_b200.scoring import Fp8Scorer

    H, V, rows = 512, 3000, 30
    g = torch.Generator().manual_seed(4)
    n = AddRMSNorm(H, device="cuda")
    b = None if bias is None else (torch.randn(V, generator=g) * 3).to(DT[bias]).cuda()
    w = (torch.randn(V, H, generator=g) * 0.4).bfloat16().cuda()  # logits of 9 and more
    head = Fp8Head(w, b, out_dtype=DT[head_dtype])
    x, r = (torch.randn(rows, H, generator=g).bfloat16().cuda() for _ in range(2))
    t = torch.randint(0, V, (rows,), generator=g).cuda()
    out = Fp8Scorer(n, head, block_rows=16)(x, r, t)
    q, s, _ = n.quantized(x, r)
    z, mag = o.block_matmul(_np(q.float()), _np(s), _np(head.codes.float()), _np(head.scale),
                            _np(b))
    want = o.token_logprobs(z, t.cpu().numpy())
    # the product: 128 + 8 roundings of a step within a block, then its scales and
    # the blocks' sum, each of the magnitudes at most
    dz = ((mag + (0 if b is None else np.abs(_np(b)))) * 2 * (136 + 8) * U).max()
    assert 2 * dz < 0.01  # (bf16 logits of 16 are off by up to 0.06)
    _close(_np(out["logp"]), want["logp"], 2 * dz + 4 * tol(V))
    _close(_np(out["entropy"]), want["entropy"], 2 * dz * (2 + np.log(V)) + 30 * tol(V))
    # the head itself answers in its own type, and in another on request
    zh = head.logits(q, s)
    assert zh.dtype == DT[head_dtype]
    z32 = head.logits(q, s, out_dtype=torch.float32)
    assert z32.dtype == torch.float32
    _close(_np(z32), z, dz)
    if b is None or bias == head_dtype:
        assert torch.equal(zh, z32.to(DT[head_dtype]))


# ------------------------------------------------ what is written over, and autograd
def test_a_backward_that_saved_what_was_overwritten_raises():
    """The residual of an in-place norm and the ``out`` of a product count as
    changed, views of them too."""
    from lm_head_projection_b200 import fp8, norm

    x, w = torch.randn(4, 64, device="cuda"), torch.ones(64, device="cuda")
    r = torch.randn(4, 64, device="cuda")
    a = torch.ones(4, 64, device="cuda", requires_grad=True)
    y = (a * r).sum()  # saves r
    norm.add_rms_norm(x, w, r, inplace=True)
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        y.backward()
    qa, sa, qb, sb = _product_inputs(4, 8, 64)
    buf = torch.randn(6, 8, device="cuda")
    b = torch.ones(6, 8, device="cuda", requires_grad=True)
    y = (b * buf).sum()
    fp8.block_matmul(qa, sa, qb, sb, out_dtype=torch.float32, out=buf[1:5])
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        y.backward()
    # not given, nothing counts
    y = (b * buf).sum()
    fp8.block_matmul(qa, sa, qb, sb)
    norm.add_rms_norm(x, w, r)
    y.backward()
    with torch.inference_mode():  # tensors without a version
        r2 = torch.randn(4, 64, device="cuda")
        h = (x + r2).clone()
        assert torch.equal(norm.add_rms_norm(x, w, r2, inplace=True)["H"], h)
        assert torch.equal(r2, h)


def test_writing_over_given_tensors_inside_a_graph():
    from lm_head_projection_b200 import fp8, norm

    x, w = torch.randn(4, 64, device="cuda"), torch.ones(64, device="cuda")
    r0 = torch.randn(4, 64, device="cuda")
    r = r0.clone()
    qa, sa, qb, sb = _product_inputs(4, 8, 64)
    d = torch.zeros(4, 8, device="cuda", dtype=torch.bfloat16)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        norm.add_rms_norm(x, w, r, inplace=True)
        fp8.block_matmul(qa, sa, qb, sb, out=d)
    r.copy_(r0)
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(r, x + r0) and torch.equal(d, fp8.block_matmul(qa, sa, qb, sb))


def test_a_head_in_a_model_that_is_cast_and_moved():
    """The uncast head's bits after .to(dtype), a trip to the host and a new
    head's load_state_dict."""
    from lm_head_projection_b200.fp8 import Fp8Head

    w = (torch.randn(1000, 256) * 0.05).cuda()
    b = torch.randn(1000).cuda()
    x = torch.randn(9, 256).bfloat16().cuda()
    head = Fp8Head(w, b)
    want = head(x)
    state = {k: v.clone() for k, v in head.state_dict().items()}
    model = torch.nn.Sequential(head)
    for m in (model.to(torch.bfloat16), model.half(), model.cpu().cuda(), model.float()):
        assert torch.equal(m(x), want)
    other = Fp8Head(torch.zeros_like(w), torch.zeros_like(b))
    other.load_state_dict(state)
    assert torch.equal(other(x), want)


def test_one_row_without_leading_dimensions():
    """``[H]`` in, a number (or ``[top_k]``) out, as the shapes say."""
    from lm_head_projection_b200 import fp8
    from lm_head_projection_b200.norm import AddRMSNorm
    from lm_head_projection_b200.scoring import Fp8Scorer

    H, V = 256, 700
    n = AddRMSNorm(H, device="cuda")
    head = fp8.Fp8Head((torch.randn(V, H) * 0.1).cuda())
    x, r = (torch.randn(3, H).bfloat16().cuda() for _ in range(2))
    t = torch.tensor([5, 6, 7]).cuda()
    sc = Fp8Scorer(n, head, top_k=4)
    want = sc(x, r, t)
    one = sc(x[1], r[1], t[1])
    assert one["logp"].shape == one["entropy"].shape == () and one["top_ids"].shape == (4,)
    assert one["H"].shape == (H,)
    for k in want:
        assert torch.equal(one[k], want[k][1]), k
    q, s = fp8.quantize_rows(x[1])
    assert q.shape == (H,) and s.shape == (2,)
    assert torch.equal(head(x[1]), head(x)[1]) and head(x[1]).shape == (V,)


# ------------------------------------------------ deep products, block by block
def _blockwise(qa, sa, qb, sb):
    """In 64 bits: the product, and how far fp32 may be off.  A block's 128 products
    are exact and added in at most 128 + 8 steps of up to 2 U (the tensor cores may
    cut) of their magnitudes' sum; its scales' product and its addition are off by U
    each of the result and of the sum so far, which the blocks' magnitudes bound."""
    M, K = qa.shape
    N = qb.shape[0]
    d, inner, outer = (torch.zeros(M, N, dtype=torch.float64, device="cuda") for _ in range(3))
    per_row = sb.double().repeat_interleave(128, 0)[:N]
    nb = sa.shape[1]
    for j in range(nb):
        a = qa[:, 128 * j:128 * j + 128].double() * sa[:, j:j + 1].double()
        b = qb[:, 128 * j:128 * j + 128].double() * per_row[:, j:j + 1]
        p = a @ b.T
        d += p
        outer += p.abs()
        inner += a.abs() @ b.abs().T
    return d, 2 * (128 + 8) * U * inner + 2 * (nb + 2) * U * outer


@pytest.mark.parametrize("M,N,K", [
    (3, 9601, 67216),                    # too deep for the small kernel: pairs of 3 tokens
    (1, 300, 14336), (16, 1000, 14352), (40, 20000, 8208),   # small kernel, 16 to 64 columns
    (129, 300, 14320), (300, 2600, 8208), (1000, 2504, 4112)])
def test_deep_products_lose_no_block(M, N, K):
    """Every eighth block of K in turn weighs 256 times the others, the short last
    one among them: whole outputs, to a bound that any lost block exceeds."""
    from lm_head_projection_b200 import fp8

    qa, sa, qb, sb = _product_inputs(M, N, K)
    nb = sa.shape[1]
    j = torch.arange(nb, device="cuda")
    for p in range(8):
        s = torch.where((j % 8 == p) | (j == nb - 1), 256.0, 1.0) * sa
        want, bound = _blockwise(qa, s, qb, sb)
        got = fp8.block_matmul(qa, s, qb, sb, out_dtype=torch.float32).double()
        err = (got - want).abs()
        assert (err <= bound + want.abs() * U).all(), (p, (err / bound).max())
        # what one heavy block adds, the smallest of them, is above the bound
        k0 = 128 * (nb - 1)
        tail = (qa[:, k0:].double() * s[:, -1:].double()) @ (
            qb[:, k0:].double() * sb.double().repeat_interleave(128, 0)[:N, -1:]).T
        assert tail.square().mean().sqrt() > 4 * bound.mean()


# ------------------------------------------- norm backwards on a stream of their own
def test_norm_backwards_allocate_on_the_stream_they_are_given():
    """Their workspace is freed on return, while the kernels run: it must not go back
    to the current stream, which is busy allocating the same size."""
    from lm_head_projection_b200 import flkl_norm_workspace_size, norm

    g = torch.Generator(device="cuda").manual_seed(2)
    x, dy = (torch.randn(4096, 2048, device="cuda", generator=g) for _ in range(2))
    w = torch.randn(2048, device="cuda", generator=g)
    want = [norm.rms_norm_backward(dy, x, w), norm.layer_norm_backward(dy, x, w)]
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    for _ in range(5):
        got = [norm.rms_norm_backward(dy, x, w, stream=side),
               norm.layer_norm_backward(dy, x, w, stream=side)]
        for n in (1, 2):
            torch.full((flkl_norm_workspace_size(4096, 2048, True, n == 2),), 0xFF,
                       dtype=torch.uint8, device="cuda")
        side.synchronize()
        for a, b in zip(got, want):
            for k in a:
                assert a[k] is None or torch.equal(a[k], b[k]), k
    torch.cuda.synchronize()


# --------------------------------------------------------------- the chain's ends
def test_scorer_without_rows_and_captured_with_a_bias():
    from lm_head_projection_b200.fp8 import Fp8Head
    from lm_head_projection_b200.norm import AddRMSNorm
    from lm_head_projection_b200.scoring import Fp8Scorer

    H, V = 256, 1000
    n = AddRMSNorm(H, device="cuda")
    head = Fp8Head((torch.randn(V, H) * 0.1).cuda(), torch.randn(V).bfloat16().cuda())
    sc = Fp8Scorer(n, head, top_k=3, block_rows=16)
    for lead in ((0,), (2, 0)):
        out = sc(torch.empty(*lead, H).bfloat16().cuda(), None,
                 torch.empty(lead, dtype=torch.int64, device="cuda"))
        assert out["logp"].shape == lead and out["top_ids"].shape == (*lead, 3)
    x = torch.randn(40, H).bfloat16().cuda()
    t = torch.randint(0, V, (40,)).cuda()
    want = sc(x, None, t)
    xs = torch.randn_like(x)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out = sc(xs, None, t)
    xs.copy_(x)
    g.replay()
    torch.cuda.synchronize()
    for k in ("logp", "entropy", "top_logp", "top_ids"):
        assert torch.equal(out[k], want[k]), k
    with pytest.raises(ValueError, match="out"):
        head.logits(*n.quantized(x)[:2], out=torch.empty(40, V, device="cuda"))
