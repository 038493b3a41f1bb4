"""The operators of the scoring path behind a vocabulary head, as they are measured.

Three operators that follow one another where a model answers or is scored,
the first and the last of them with their gradients where it trains:

* ``norm_fp8`` / ``norm`` / ``norm_train``: the residual's addition and the
  root-mean-square norm, with an output in e4m3 and one scale per row and 128
  columns, with an output of the input's type, or with that output and the
  backward pass;
* ``matmul``: the product of two e4m3 matrices whose scales stand per row and
  128 columns (activations) and per 128 x 128 block (weights);
* ``logprob`` / ``logprob_train``: log-probabilities of given tokens, the
  entropy and the best alternatives of rows of logits, and the gradient.

``run`` computes them in plain torch operations (``own`` false) or through
``lm_head_projection_b200`` (``own`` true).
"""

import math

import torch

own = False

IGNORE = -100
E4M3_MAX = 448.0
EPS = 1e-6
DTYPES = {"bf16": torch.bfloat16, "fp32": torch.float32}


def listed():
    return [
        # the last norm before the head while a few sequences are answered
        dict(name="norm_fp8_8x4096", op="norm_fp8", rows=8, H=4096, dtype="bf16"),
        # the same over a long prompt, the widest rows
        dict(name="norm_fp8_8192x8192", op="norm_fp8", rows=8192, H=8192, dtype="bf16"),
        # a norm layer of a training step, forward and backward
        dict(name="norm_train_4096x8192", op="norm_train", rows=4096, H=8192, dtype="bf16"),
        # the same in fp32, sizes that fill no tile
        dict(name="norm_train_fp32_999x2056", op="norm_train", rows=999, H=2056, dtype="fp32"),
        # the head for one new token: the weight is read once
        dict(name="matmul_1x128256x4096", op="matmul", M=1, N=128256, K=4096, out="bf16"),
        # a projection in front of the head for a batch of new tokens: latency
        dict(name="matmul_40x4096x4096", op="matmul", M=40, N=4096, K=4096, out="fp32"),
        # the head over a scored batch: the tensor cores' rate
        dict(name="matmul_1024x128256x4096", op="matmul", M=1024, N=128256, K=4096, out="bf16"),
        # rows, columns and depth that fill no tile, rows of the output unaligned
        dict(name="matmul_777x50257x1552", op="matmul", M=777, N=50257, K=1552, out="bf16"),
        # sampling four tokens with alternatives, part of the vocabulary masked
        dict(name="logprob_4x128256", op="logprob", rows=4, V=128256, pad=0, dtype="bf16", k=20,
             T=0.7, mask="inf", ignore=0.0),
        # scoring a batch of given tokens, a tenth of the rows is padding
        dict(name="logprob_2048x128256", op="logprob", rows=2048, V=128256, pad=0, dtype="bf16",
             k=5, T=1.0, mask="", ignore=0.1),
        # a policy step: log-probabilities and entropy with their gradient
        dict(name="logprob_train_1024x151936", op="logprob_train", rows=1024, V=151936, pad=0,
             dtype="bf16", k=0, T=1.0, mask="", ignore=0.1),
        # fp32 logits of an odd vocabulary in padded rows, masked with the lowest value
        dict(name="logprob_train_fp32_37x50257", op="logprob_train", rows=37, V=50257, pad=47,
             dtype="fp32", k=32, T=1.3, mask="lowest", ignore=0.1),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["norm_fp8", "norm", "norm_train", "matmul", "matmul", "logprob", "logprob",
                     "logprob_train"])
    if op.startswith("norm"):
        H = 8 * _log_int(rng, 8, 1024)
        most = (4096 if op == "norm_train" else 8192) * 8192
        return dict(op=op, rows=_log_int(rng, 1, min(16384, most // H)), H=H,
                    dtype=rng.choice(["bf16", "bf16", "fp32"]))
    if op == "matmul":
        K = 16 * _log_int(rng, 8, 512)
        N = _log_int(rng, 64, 151936)
        most = min(4096, 1024 * 128256 * 4096 // (N * K))
        return dict(op=op, M=_log_int(rng, 1, max(1, most)), N=N, K=K,
                    out=rng.choice(["bf16", "bf16", "fp32"]))
    V = _log_int(rng, 1000, 151936)
    most = (1024 * 151936 if op == "logprob_train" else 2048 * 128256) // (V + 64)
    dtype = rng.choice(["bf16", "bf16", "fp32"])
    return dict(op=op, rows=_log_int(rng, 1, min(4096, most // (2 if dtype == "fp32" else 1))),
                V=V, pad=rng.choice([0, 0, rng.randint(1, 64)]), dtype=dtype,
                k=rng.choice([0, 1, 5, 8, 20, 32]), T=rng.choice([1.0, 0.6, 1.3]),
                mask=rng.choice(["", "inf", "lowest"]), ignore=rng.choice([0.0, 0.1]))


# ------------------------------------------------------------------ inputs

def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _randn(g, *shape):
    return torch.randn(shape, generator=g, device="cuda")


def _group_scales(x, rows, cols):
    """Largest magnitude / 448 of each rows x cols block of x (1 where a block is 0)."""
    n, k = x.shape
    a = torch.nn.functional.pad(x.abs(), (0, -k % cols, 0, -n % rows))
    a = a.view(a.shape[0] // rows, rows, a.shape[1] // cols, cols).amax((1, 3))
    return torch.where(a > 0, a / E4M3_MAX, torch.ones_like(a))


def _spread(scale, n, k, rows, cols):
    return scale.repeat_interleave(rows, 0)[:n].repeat_interleave(cols, 1)[:, :k]


def _quantized(x, rows, cols):
    s = _group_scales(x, rows, cols)
    q = x.div_(_spread(s, *x.shape, rows, cols)).clamp_(-E4M3_MAX, E4M3_MAX)
    return q.to(torch.float8_e4m3fn), s


def prepare(case, seed):
    g = _gen(seed)
    if case["op"].startswith("norm"):
        rows, H, dt = case["rows"], case["H"], DTYPES[case["dtype"]]
        s = dict(op=case["op"], W=(1 + 0.1 * _randn(g, H)).to(dt))
        # a few channels of the residual stream are far larger than the rest
        channel = 1 + 15 * (torch.rand(H, generator=g, device="cuda") < 0.01)
        s["residual"] = (_randn(g, rows, H) * channel).to(dt)
        s["X"] = _randn(g, rows, H).to(dt)
        if case["op"] == "norm_train":
            s["dY"] = _randn(g, rows, H).to(dt)
            s["dH"] = _randn(g, rows, H).to(dt)
        return s
    if case["op"] == "matmul":
        M, N, K = case["M"], case["N"], case["K"]
        A, a_scale = _quantized(_randn(g, M, K) * torch.exp(_randn(g, M, 1)), 1, 128)
        B, b_scale = _quantized(_randn(g, N, K) * 0.02, 128, 128)
        return dict(op="matmul", A=A, a_scale=a_scale, B=B, b_scale=b_scale,
                    out=DTYPES[case["out"]])
    rows, V, dt = case["rows"], case["V"], DTYPES[case["dtype"]]
    z = _randn(g, rows, V + case["pad"]).mul_(2.0)
    target = torch.randint(0, V, (rows,), generator=g, device="cuda")
    z.scatter_add_(1, target[:, None], 12 * torch.rand((rows, 1), generator=g, device="cuda"))
    if case["mask"]:
        low = -math.inf if case["mask"] == "inf" else torch.finfo(dt).min
        keep = torch.rand(z.shape, generator=g, device="cuda") < 0.5
        keep.scatter_(1, target[:, None], True)
        if rows > 2:
            keep[rows // 2] = False  # a row whose mask leaves nothing
        z.masked_fill_(~keep, low)
        del keep
    z = z.to(dt)[:, :V]
    dropped = torch.rand(rows, generator=g, device="cuda") < case["ignore"]
    target = torch.where(dropped, IGNORE, target)
    s = dict(op=case["op"], logits=z, target=target, T=case["T"], k=case["k"])
    if case["op"] == "logprob_train":
        s["dlogp"] = _randn(g, rows)
        s["dentropy"] = _randn(g, rows) * 0.01
        s["dtop"] = _randn(g, rows, case["k"]) * 0.1 if case["k"] else None
    return s


# ------------------------------------------------------------------ plain forms

def _plain_norm(s):
    dt = s["X"].dtype
    H = (s["X"].float() + s["residual"].float()).to(dt)  # the residual stream, as it is kept
    h, w = H.float(), s["W"].float()
    r = 1 / torch.sqrt((h * h).mean(1, keepdim=True) + EPS)
    y = h * r * w
    if s["op"] == "norm_fp8":
        scale = _group_scales(y, 1, 128)
        q = (y / _spread(scale, *y.shape, 1, 128)).clamp(-E4M3_MAX, E4M3_MAX)
        return {"Y": q.to(torch.float8_e4m3fn), "scale": scale, "H": H}
    out = {"Y": y.to(dt), "H": H}
    if s["op"] == "norm_train":
        dy, xhat = s["dY"].float(), h * r
        gw = dy * w
        dx = s["dH"].float() + (gw - xhat * (gw * xhat).mean(1, keepdim=True)) * r
        out["dX"] = dx.to(dt)
        out["dW"] = (dy * xhat).sum(0)
    return out


def _plain_matmul(s):
    a = s["A"].float() * _spread(s["a_scale"], *s["A"].shape, 1, 128)
    b = s["B"].float() * _spread(s["b_scale"], *s["B"].shape, 128, 128)
    return (a @ b.t()).to(s["out"])


def _order(z):
    """int64 keys of fp32 values that sort as (value, lower index first)."""
    bits = (z + 0.0).view(torch.int32)
    bits = torch.where(bits < 0, bits ^ 0x7FFFFFFF, bits).long()
    return bits * 2**32 + torch.arange(z.shape[1] - 1, -1, -1, device=z.device)


def _plain_logprob(s):
    z, target, T, k = s["logits"].float(), s["target"], s["T"], s["k"]
    V = z.shape[1]
    kept = target != IGNORE
    m = z.amax(1)
    full = m > -math.inf  # rows that hold any token
    u = (z - torch.where(full, m, 0.0)[:, None]) / T
    e = torch.exp(u)
    total = e.sum(1)
    eu = torch.where(e > 0, e * u, 0.0).sum(1)
    ln = torch.log(torch.where(full, total, 1.0))
    entropy = torch.where(full & kept, ln - eu / torch.where(full, total, 1.0), 0.0)
    lse = torch.where(full, m / T + ln, -math.inf)
    picked = u.gather(1, target.clamp(0, V - 1)[:, None])[:, 0] - ln
    logp = torch.where(kept, torch.where(full, picked, -math.inf), 0.0)
    out = {"logp": logp, "entropy": entropy, "lse": torch.where(kept, lse, 0.0)}
    if k:
        ids = _order(z).topk(k, 1).indices
        top = u.gather(1, ids) - ln[:, None]
        top = torch.where(full[:, None], top, -math.inf)
        out["top_logp"] = torch.where(kept[:, None], top, 0.0)
        out["top_ids"] = torch.where(kept[:, None], ids, -1)
    if s["op"] == "logprob_train":
        logq = u - ln[:, None]
        p = e / torch.where(full, total, 1.0)[:, None]
        gl = s["dlogp"]
        coef = gl.clone()
        if k:
            gt = s["dtop"]
            coef = coef + gt.sum(1)
        d = -coef[:, None] * p
        d = d - torch.where(p > 0, s["dentropy"][:, None] * p * (logq + entropy[:, None]), 0.0)
        d.scatter_add_(1, target.clamp(0, V - 1)[:, None], gl[:, None])
        if k:
            d.scatter_add_(1, ids, gt)
        d = torch.where((kept & full)[:, None], d / T, 0.0)
        out["dlogits"] = d.to(s["logits"].dtype)
    return out


# ------------------------------------------------------------------ one pass

def _own(s):
    from lm_head_projection_b200 import fp8, logprobs, norm

    if s["op"].startswith("norm"):
        r = norm.add_rms_norm(s["X"], s["W"], s["residual"], eps=EPS,
                              quantize=s["op"] == "norm_fp8")
        if s["op"] == "norm_fp8":
            return {"Y": r["Y"], "scale": r["scale"], "H": r["H"]}
        out = {"Y": r["Y"], "H": r["H"]}
        if s["op"] == "norm_train":
            b = norm.add_rms_norm_backward(s["dY"], r["H"], s["W"], dH=s["dH"], eps=EPS)
            out["dX"], out["dW"] = b["dX"], b["dW"]
        return out
    if s["op"] == "matmul":
        return fp8.block_matmul(s["A"], s["a_scale"], s["B"], s["b_scale"], out_dtype=s["out"])
    r = logprobs.token_logprobs_forward(s["logits"], s["target"], ignore_index=IGNORE,
                                        temperature=s["T"], top_k=s["k"])
    out = {n: r[n] for n in ("logp", "entropy", "lse")}
    if s["k"]:
        out["top_logp"], out["top_ids"] = r["top_logp"], r["top_ids"]
    if s["op"] == "logprob_train":
        out["dlogits"] = logprobs.token_logprobs_backward(
            s["logits"], s["target"], r, dlogp=s["dlogp"], dentropy=s["dentropy"],
            dtop_logp=s["dtop"], ignore_index=IGNORE, temperature=s["T"])
    return out


def run(state):
    if own:
        return _own(state)
    if state["op"].startswith("norm"):
        return _plain_norm(state)
    if state["op"] == "matmul":
        return _plain_matmul(state)
    return _plain_logprob(state)


def work(case):
    if case["op"].startswith("norm"):
        n, H = case["rows"] * case["H"], case["H"]
        e = 2 if case["dtype"] == "bf16" else 4
        if case["op"] == "norm_fp8":  # x, residual, the new residual, codes and scales
            return {"bytes": n * (3 * e + 1) + case["rows"] * -(-H // 128) * 4 + H * e,
                    "flops": 8 * n}
        if case["op"] == "norm":
            return {"bytes": n * 4 * e + H * e, "flops": 5 * n}
        # x, residual, dY, dH in; y, the new residual, dX and dW out
        return {"bytes": n * 8 * e + H * (e + 4), "flops": 16 * n}
    if case["op"] == "matmul":
        M, N, K = case["M"], case["N"], case["K"]
        kb = -(-K // 128)
        out = 2 if case["out"] == "bf16" else 4
        return {"bytes": (M + N) * K + 4 * kb * (M + -(-N // 128)) + M * N * out,
                "flops": 2 * M * N * K}
    rows, V, k = case["rows"], case["V"], case["k"]
    e = 2 if case["dtype"] == "bf16" else 4
    kept = rows * (1 - case["ignore"])
    small = rows * (8 + 3 * 4 + 12 * k)
    if case["op"] == "logprob":
        return {"bytes": kept * V * e + small, "flops": 6 * kept * V}
    # logits in, their gradient out (dropped rows are written as zeros)
    return {"bytes": (kept + rows) * V * e + small + rows * (8 + 4 * k), "flops": 13 * kept * V}


# ------------------------------------------------------------------ in 64 bits

def _exact_norm(s):
    dt = s["X"].dtype
    h = (s["X"].double() + s["residual"].double()).to(torch.float32).to(dt).double()
    w = s["W"].double()
    rms = (h.square().sum(1, keepdim=True) / h.shape[1] + EPS).sqrt()
    y = h / rms * w
    if s["op"] == "norm_fp8":
        blocks = [c.abs().amax(1) / E4M3_MAX for c in y.split(128, 1)]
        scale = torch.stack([torch.where(c > 0, c, 1.0) for c in blocks], 1)
        codes = [c / scale[:, i:i + 1] for i, c in enumerate(y.split(128, 1))]
        return {"Y": torch.cat(codes, 1), "scale": scale, "H": h}
    out = {"Y": y, "H": h}
    if s["op"] == "norm_train":
        g = s["dY"].double() * w
        dot = (g * h).sum(1, keepdim=True) / h.shape[1]
        out["dX"] = s["dH"].double() + g / rms - h * dot / rms**3
        out["dW"] = (s["dY"].double() * h / rms).sum(0)
    return out


def _exact_matmul(s):
    M, K = s["A"].shape
    N = s["B"].shape[0]
    total = torch.zeros((M, N), dtype=torch.float64, device="cuda")
    per_block = s["b_scale"].double().repeat_interleave(128, 0)[:N]
    for i, k0 in enumerate(range(0, K, 128)):
        a = s["A"][:, k0:k0 + 128].double() * s["a_scale"][:, i:i + 1].double()
        b = s["B"][:, k0:k0 + 128].double() * per_block[:, i:i + 1]
        total.addmm_(a, b.t())
    return total


def _exact_logprob(s):
    """Row by row, from log_softmax's definition in 64 bits."""
    k, T = s["k"], s["T"]
    names = ["logp", "entropy", "lse"] + (["top_logp", "top_ids"] if k else [])
    rows, V = s["logits"].shape
    train = s["op"] == "logprob_train"
    got = {n: [] for n in names}
    grads = torch.zeros((rows, V), dtype=torch.float64, device="cuda") if train else None
    targets = s["target"].tolist()
    zero = torch.zeros((), dtype=torch.float64, device="cuda")
    for r, t in enumerate(targets):
        z = s["logits"][r].double()
        if t == IGNORE:
            row = dict(logp=zero, entropy=zero, lse=zero,
                       top_logp=zero.expand(k), top_ids=torch.full((k,), -1, device="cuda"))
        else:
            top = z.max()  # taken off first: the lowest value of a type swallows ln V
            empty = top == -math.inf
            u = torch.where(empty, -math.inf, z - torch.where(empty, 0.0, top)) / T
            logq = torch.where(empty, u, u - torch.logsumexp(u, 0))
            p = logq.exp()
            entropy = -torch.where(p > 0, p * logq, 0.0).sum()
            row = dict(logp=logq[t], entropy=entropy, lse=top / T + torch.logsumexp(u, 0))
            if k:
                row["top_ids"] = torch.sort(z, descending=True, stable=True).indices[:k]
                row["top_logp"] = logq[row["top_ids"]]
            if train:
                gl, ge = s["dlogp"][r].double(), s["dentropy"][r].double()
                d = -gl * p - ge * torch.where(p > 0, p * (logq + entropy), 0.0)
                d[t] += gl
                if k:
                    gt = s["dtop"][r].double()
                    d -= gt.sum() * p
                    d[row["top_ids"]] += gt
                grads[r] = torch.where(empty, 0.0, d / T)
        for n in names:
            got[n].append(row[n])
    out = {n: torch.stack(v) for n, v in got.items()}
    if train:
        out["dlogits"] = grads
    return out


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"].startswith("norm"):
        return _exact_norm(s)
    if case["op"] == "matmul":
        return _exact_matmul(s)
    return _exact_logprob(s)
