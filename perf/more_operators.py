"""Products with a full epilogue, and products grouped by expert, as they are
measured.  Each kind of case below is one operator through
`dense_gemm_tiled_gb300.binding`, and a plain form of elementary torch
operations in 32 bits:

  fused      U = A B^T + bias,  Y = act(U) + R          (U kept for the backward
             pass where the case says so)
  fused_bwd  dX = (A B) act'(U),  dbias = column sums of dX
  grouped    `fused` for rows o[e] .. o[e+1] of A with B[e] and bias[e]
  grouped_bwd  `fused_bwd` likewise, dbias[e] for each group
  wgrad      C[e] = A_e^T B_e over the rows of group e

Group e's rows are o[e] .. o[e+1] of the row dimension; the offsets lie on the
GPU, as a router leaves them.  The buffers hold `pad` rows behind the last
group, which nothing touches.
"""
import math

import torch

own = False

DT = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}


# ---------------------------------------------------------------------------
# The cases
# ---------------------------------------------------------------------------
def listed():
    return [
        # one new token through an MLP's up projection: latency
        dict(name="fused 1x5632x2048 bf16", op="fused", M=1, N=5632, K=2048, dtype="bf16",
             act="gelu", bias=True, residual=False, preact=False),
        # the LoRA step's down projection, added to the residual stream
        dict(name="fused 512x2048x5632 f16", op="fused", M=512, N=2048, K=5632, dtype="f16",
             act="none", bias=True, residual=True, preact=False),
        # the largest square of the sweep in training: everything the epilogue does
        dict(name="fused 8192^3 bf16", op="fused", M=8192, N=8192, K=8192, dtype="bf16",
             act="gelu", bias=True, residual=True, preact=True),
        # ragged fp32: no size a multiple of anything the kernels use
        dict(name="fused 1000x3001x777 f32", op="fused", M=1000, N=3001, K=777, dtype="f32",
             act="relu", bias=True, residual=True, preact=False),
        # the LoRA step's gradient through the down projection and the activation
        dict(name="fused_bwd 512x5632x2048 f16", op="fused_bwd", M=512, N=5632, K=2048,
             dtype="f16", act="gelu"),
        # the same at the length of a long-context batch
        dict(name="fused_bwd 16384x5632x2048", op="fused_bwd", M=16384, N=5632, K=2048,
             dtype="bf16", act="gelu"),
        # a small serving batch: 16 tokens, two experts each, of 64; bound by the
        # weights of the experts that have rows
        dict(name="grouped decode 32 rows of 64", op="grouped", T=32, groups=64, empty=40,
             pad=0, N=1408, K=2048, dtype="bf16", act="gelu", bias=True, residual=False,
             preact=False),
        # a training batch over eight experts, their sizes uneven, one of them empty
        dict(name="grouped 4000 rows of 8", op="grouped", T=4000, groups=8, empty=1, pad=96,
             N=5632, K=2048, dtype="bf16", act="gelu", bias=True, residual=False, preact=True),
        # the gradient through those experts' down projection and activation
        dict(name="grouped_bwd 4000 rows of 8", op="grouped_bwd", T=4000, groups=8, empty=1,
             pad=96, N=5632, K=2048, dtype="bf16", act="gelu"),
        # many small experts at a long-context batch's length
        dict(name="grouped_bwd 32768 rows of 64", op="grouped_bwd", T=32768, groups=64, empty=0,
             pad=0, N=1408, K=2048, dtype="f16", act="gelu"),
        # the weight gradients of both
        dict(name="wgrad 4000 rows of 8", op="wgrad", T=4000, groups=8, empty=1, pad=96, M=5632,
             N=2048, dtype="bf16"),
        dict(name="wgrad 32768 rows of 64", op="wgrad", T=32768, groups=64, empty=0, pad=0,
             M=1408, N=2048, dtype="f16"),
    ]


def _size(rng, lo, hi):
    """A size of [lo, hi], spread over the logarithm; one in two odd or ragged,
    the others multiples of 80 where that fits."""
    v = int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))
    if v >= 160 and rng.random() < 0.5:
        v = v // 80 * 80
    return max(lo, min(hi, v))


def draw(rng):
    op = rng.choice(["fused", "fused_few", "fused_bwd", "grouped", "grouped_few", "grouped_bwd",
                     "wgrad"])
    dtype = rng.choice(["f16", "bf16", "f16", "bf16", "f32"])
    top = 4096 if dtype == "f32" else 8192
    act = rng.choice(["none", "relu", "gelu"])
    extra = dict(bias=rng.random() < 0.7, residual=rng.random() < 0.5)
    if op in ("fused", "fused_few"):
        few = op == "fused_few"
        return dict(op="fused", M=_size(rng, 1, 32) if few else _size(rng, 33, top),
                    N=_size(rng, 32, top), K=_size(rng, 32, top), dtype=dtype, act=act,
                    preact=rng.random() < 0.4, **extra)
    if op == "fused_bwd":
        return dict(op=op, M=_size(rng, 1, top), N=_size(rng, 32, top), K=_size(rng, 32, 4096),
                    dtype=dtype, act=rng.choice(["relu", "gelu"]))
    groups = _size(rng, 1, 64)
    few = op == "grouped_few"
    T = _size(rng, 1, 64) if few else _size(rng, 64, 2 * top)
    c = dict(T=T, groups=groups, empty=rng.randint(0, groups // 2), pad=rng.choice([0, 1, 50]),
             dtype=dtype)
    if op == "wgrad":
        return dict(op=op, M=_size(rng, 32, 2048), N=_size(rng, 32, 2048), **c)
    c.update(N=_size(rng, 32, 2048), K=_size(rng, 32, 2048))
    if op == "grouped_bwd":
        return dict(op=op, act=rng.choice(["relu", "gelu"]), **c)
    return dict(op="grouped", act=act, preact=not few and rng.random() < 0.4, **extra, **c)


def _sizes(c):
    """Rows of each group before the seed shuffles them: `empty` groups without
    any (at least one group has rows), the others in proportion to 1 / (rank + 2)
    and at least one row each while there are enough."""
    live = max(1, min(c["groups"] - c["empty"], c["T"]))
    share = [1.0 / (r + 2) for r in range(live)]
    total = sum(share)
    n = [1 + int((c["T"] - live) * s / total) for s in share]
    n[0] += c["T"] - sum(n)
    return n + [0] * (c["groups"] - live)


# ---------------------------------------------------------------------------
# Inputs
# ---------------------------------------------------------------------------
def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _normal(g, shape, std, dtype):
    return (torch.randn(shape, generator=g, device="cuda") * std).to(DT[dtype])


def prepare(case, seed):
    """Activations and gradients ~ N(0, 1), weights ~ N(0, 0.02^2), as the LoRA
    step's; the buffers that the program writes into (zeros: rows behind the
    last group keep them)."""
    g = _gen(seed)
    c = dict(case)
    dt = c["dtype"]
    if c["op"].startswith("fused"):
        M, N, K = c["M"], c["N"], c["K"]
        rows, lead = M, ()
    else:
        order = torch.randperm(c["groups"], generator=torch.Generator().manual_seed(seed)).tolist()
        n = _sizes(c)
        n = [n[i] for i in order]
        at = [0]
        for v in n:
            at.append(at[-1] + v)
        c["at"] = at                 # the host's copy: the plain form loops over it
        c["offsets"] = torch.tensor(at, dtype=torch.int32, device="cuda")
        rows, lead = c["T"] + c["pad"], (c["groups"],)
        if c["op"] == "wgrad":
            c["A"] = _normal(g, (rows, c["M"]), 1.0, dt)
            c["B"] = _normal(g, (rows, c["N"]), 1.0, dt)
            c["C"] = torch.zeros((*lead, c["M"], c["N"]), dtype=DT[dt], device="cuda")
            return c
        N, K = c["N"], c["K"]
    backward = c["op"].endswith("bwd")
    c["A"] = _normal(g, (rows, K), 1.0, dt)
    c["B"] = _normal(g, (*lead, K, N) if backward else (*lead, N, K), 0.02, dt)
    c["Y"] = torch.zeros((rows, N), dtype=DT[dt], device="cuda")
    c["U"] = c["R"] = c["b"] = None
    if backward:
        c["U"] = _normal(g, (rows, N), 1.0, dt)
        c["db"] = torch.zeros((*lead, N), dtype=torch.float32, device="cuda")
    else:
        if c["bias"]:
            c["b"] = _normal(g, (*lead, N), 0.1, dt)
        if c["residual"]:
            c["R"] = _normal(g, (rows, N), 1.0, dt)
        if c["preact"]:
            c["U"] = torch.zeros((rows, N), dtype=DT[dt], device="cuda")
    return c


# ---------------------------------------------------------------------------
# One pass
# ---------------------------------------------------------------------------
def run(state):
    return (_run_own if own else _run_plain)(state)


def _run_plain(c):
    fp32_products = torch.backends.cuda.matmul.allow_tf32
    torch.backends.cuda.matmul.allow_tf32 = False
    try:
        return _plain(c)
    finally:
        torch.backends.cuda.matmul.allow_tf32 = fp32_products


def _act(u, act):
    if act == "gelu":
        return 0.5 * u * (1.0 + torch.erf(u * 0.7071067811865476))
    return torch.clamp(u, min=0.0) if act == "relu" else u


def _slope(u, act):
    if act == "gelu":
        return 0.5 * (1.0 + torch.erf(u * 0.7071067811865476)) + \
            u * torch.exp(-0.5 * u * u) * 0.3989422804014327
    return (u > 0).float()


def _forward(c, a, b, bias, r):
    u = a.float() @ b.float().t()
    if bias is not None:
        u = u + bias.float()
    y = _act(u, c["act"])
    if r is not None:
        y = y + r.float()
    return u, y


def _plain(c):
    dt = DT[c["dtype"]]
    if c["op"] == "fused":
        u, y = _forward(c, c["A"], c["B"], c["b"], c["R"])
        return (y.to(dt), u.to(dt)) if c["preact"] else y.to(dt)
    if c["op"] == "fused_bwd":
        d = (c["A"].float() @ c["B"].float()) * _slope(c["U"].float(), c["act"])
        return d.to(dt), d.sum(dim=0)
    for e, (lo, hi) in enumerate(zip(c["at"], c["at"][1:])):
        if c["op"] == "wgrad":
            c["C"][e] = (c["A"][lo:hi].float().t() @ c["B"][lo:hi].float()).to(dt)
        elif c["op"] == "grouped_bwd":
            d = (c["A"][lo:hi].float() @ c["B"][e].float()) * _slope(c["U"][lo:hi].float(), c["act"])
            c["Y"][lo:hi] = d.to(dt)
            c["db"][e] = d.sum(dim=0)
        elif hi > lo:
            u, y = _forward(c, c["A"][lo:hi], c["B"][e], None if c["b"] is None else c["b"][e],
                            None if c["R"] is None else c["R"][lo:hi])
            c["Y"][lo:hi] = y.to(dt)
            if c["preact"]:
                c["U"][lo:hi] = u.to(dt)
    if c["op"] == "wgrad":
        return c["C"]
    if c["op"] == "grouped_bwd":
        return c["Y"], c["db"]
    return (c["Y"], c["U"]) if c["preact"] else c["Y"]


def _run_own(c):
    from dense_gemm_tiled_gb300 import binding as g
    if c["op"] == "fused":
        g.gemm_fused(c["A"], c["B"], c["Y"], transB=True, bias=c["b"], act=c["act"],
                     residual=c["R"], preact=c["U"])
    elif c["op"] == "fused_bwd":
        g.gemm_fused_backward(c["A"], c["B"], c["Y"], c["U"], act=c["act"], dbias=c["db"])
    elif c["op"] == "grouped":
        g.gemm_grouped(c["A"], c["B"], c["Y"], c["offsets"], transB=True, bias=c["b"],
                       act=c["act"], residual=c["R"], preact=c["U"])
    elif c["op"] == "grouped_bwd":
        g.gemm_grouped_backward(c["A"], c["B"], c["Y"], c["offsets"], c["U"], act=c["act"],
                                dbias=c["db"])
    else:
        return g.gemm_grouped_wgrad(c["A"], c["B"], c["C"], c["offsets"])
    if c["op"].endswith("bwd"):
        return c["Y"], c["db"]
    return (c["Y"], c["U"]) if c["preact"] else c["Y"]


# ---------------------------------------------------------------------------
# What a pass cannot do without
# ---------------------------------------------------------------------------
def work(case):
    c = case
    es = 4 if c["dtype"] == "f32" else 2
    if c["op"] == "wgrad":
        return {"bytes": es * (c["T"] * (c["M"] + c["N"]) + c["groups"] * c["M"] * c["N"]),
                "flops": 2 * c["T"] * c["M"] * c["N"]}
    N, K = c["N"], c["K"]
    rows, live, groups = c.get("T", c.get("M")), 1, 1
    if "T" in c:
        live, groups = sum(1 for v in _sizes(c) if v), c["groups"]
    n = rows * K + live * N * K + rows * N
    if c["op"].endswith("bwd"):
        return {"bytes": es * (n + rows * N) + 4 * groups * N, "flops": 2 * rows * N * K}
    n += (rows * N if c["residual"] else 0) + (rows * N if c["preact"] else 0)
    return {"bytes": es * (n + (live * N if c["bias"] else 0)), "flops": 2 * rows * N * K}


# ---------------------------------------------------------------------------
# The definitions in 64 bits
# ---------------------------------------------------------------------------
def exact(case, seed):
    """Group by group on the GPU; Phi by erfc, so that it keeps its tail."""
    c = prepare(case, seed)
    phi = lambda t: 0.5 * torch.erfc(-t / math.sqrt(2.0))  # noqa: E731
    spans = list(zip(c["at"], c["at"][1:])) if "at" in c else [(0, c["M"])]
    if c["op"] == "wgrad":
        return torch.stack([torch.einsum("km,kn->mn", c["A"][lo:hi].double(),
                                         c["B"][lo:hi].double()) for lo, hi in spans])
    one = "at" not in c
    rows, N = c["Y"].shape
    Y = torch.zeros((rows, N), dtype=torch.float64, device="cuda")
    second = torch.zeros_like(Y)                 # U
    db = torch.zeros((len(spans), N), dtype=torch.float64, device="cuda")
    for e, (lo, hi) in enumerate(spans):
        if hi == lo:
            continue
        a, b = c["A"][lo:hi].double(), (c["B"] if one else c["B"][e]).double()
        if c["op"].endswith("bwd"):
            u = c["U"][lo:hi].double()
            if c["act"] == "gelu":
                s = phi(u) + u * torch.exp(-u * u / 2) / math.sqrt(2 * math.pi)
            else:
                s = (u > 0).double()
            Y[lo:hi] = torch.matmul(a, b) * s
            db[e] = Y[lo:hi].sum(dim=0)
            continue
        u = torch.matmul(a, b.transpose(0, 1))
        if c["b"] is not None:
            u = u + (c["b"] if one else c["b"][e]).double()[None, :]
        y = u * phi(u) if c["act"] == "gelu" else torch.relu(u) if c["act"] == "relu" else u
        Y[lo:hi] = y if c["R"] is None else y + c["R"][lo:hi].double()
        second[lo:hi] = u
    if c["op"].endswith("bwd"):
        return Y, db[0] if one else db
    return (Y, second) if c["preact"] else Y
