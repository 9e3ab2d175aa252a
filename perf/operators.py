"""Measured cases of the grouped and the 4-bit-weight products.

Four operators, all matrix products of an expert layer or of one linear layer:

  grouped          C[i] = act(A[i] . B[e] + bias[e])          rows i of group e
  grouped_k        C[e] = A[:, rows of e] . B[rows of e, :]    (weight gradient)
  qweight          C = A . W^T,  W[n, k] = scale[n, k / g] (q[n, k] - zero[n, k / g])
  qweight_grouped  the same with one W per group of rows

`own` false computes them with elementary torch operations in fp32; `own` true
calls the library.
"""
import math

import torch

own = False

_DT = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
_SIZE = {"bf16": 2, "f16": 2, "f32": 4}


def listed():
    return [
        # first product of an expert layer over a training batch: bias and GELU fused
        dict(name="experts forward", op="grouped", dtype="bf16", out="bf16", rows=8192, pad=0, groups=16,
             K=4096, N=4096, order="kn", skew=0.5, bias=True, act="gelu_erf"),
        # input gradient of such a layer: the weights are read transposed; odd row count, odd output width
        dict(name="experts input gradient", op="grouped", dtype="f16", out="f16", rows=4095, pad=33, groups=7,
             K=1000, N=4097, order="nk", skew=1.0, bias=False, act="none"),
        # one generation step: few tokens spread over many experts, each weight matrix read for one or two rows
        dict(name="experts decode step", op="grouped", dtype="bf16", out="bf16", rows=64, pad=0, groups=64,
             K=2048, N=1024, order="nk", skew=0.5, bias=False, act="none"),
        # a small fp32 layer, as in a reference run
        dict(name="experts forward small fp32", op="grouped", dtype="f32", out="f32", rows=1000, pad=24, groups=5,
             K=512, N=260, order="kn", skew=0.5, bias=True, act="gelu_tanh"),
        # weight gradients of a training batch, kept in fp32 for the optimiser
        dict(name="experts weight gradient", op="grouped_k", dtype="bf16", out="f32", rows=8192, pad=0, groups=16,
             M=2048, N=2048, skew=0.5),
        # a small layer's weight gradient: many short groups, some empty
        dict(name="experts weight gradient small", op="grouped_k", dtype="f16", out="f16", rows=1001, pad=23, groups=24,
             M=264, N=520, skew=1.5),
        # one token through one square linear layer: the smallest call of a generation step
        dict(name="one token 4096x4096", op="qweight", dtype="bf16", out="bf16", M=1, N=4096, K=4096, g=128, zeros=False),
        # one token through a wide linear layer, fp16 with zero points
        dict(name="one token 16384x8192", op="qweight", dtype="f16", out="f16", M=1, N=16384, K=8192, g=64, zeros=True),
        # a batch of sequences in generation, fine groups, odd width, fp32 out (logits)
        dict(name="13 tokens 4097x4352", op="qweight", dtype="bf16", out="f32", M=13, N=4097, K=4352, g=32, zeros=True),
        # a prompt
        dict(name="prompt 2048 tokens", op="qweight", dtype="bf16", out="bf16", M=2048, N=4096, K=4096, g=128, zeros=False),
        # a generation step through experts kept in 4 bits
        dict(name="4-bit experts decode step", op="qweight_grouped", dtype="bf16", out="bf16", rows=64, pad=0, groups=64,
             N=2048, K=2048, g=128, zeros=False, skew=0.5),
        # a larger batch through 4-bit experts: unequal groups, padded rows behind the last one
        dict(name="4-bit experts batch", op="qweight_grouped", dtype="f16", out="f16", rows=700, pad=68, groups=12,
             N=2056, K=1024, g=32, zeros=True, skew=1.0),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _draw(rng):
    op = rng.choice(("grouped", "grouped_k", "qweight", "qweight_grouped"))
    dtype = rng.choice(("bf16", "f16"))
    if op == "grouped":
        dtype = rng.choice(("bf16", "f16", "bf16", "f16", "f32"))
        order = rng.choice(("kn", "nk"))
        N = 8 * _log(rng, 32, 512)
        if order == "nk" and rng.random() < 0.5:
            N += rng.randrange(1, 8)
        return dict(op=op, dtype=dtype, out=dtype if rng.random() < 0.7 else "f32", rows=_log(rng, 16, 8192),
                    pad=rng.choice((0, 17)), groups=_log(rng, 4, 64), K=8 * _log(rng, 32, 512), N=N, order=order,
                    skew=rng.choice((0.0, 0.5, 1.0)), bias=rng.random() < 0.5,
                    act=rng.choice(("none", "gelu_erf", "gelu_tanh")))
    if op == "grouped_k":
        return dict(op=op, dtype=dtype, out=rng.choice(("f32", dtype)), rows=_log(rng, 256, 8192), pad=rng.choice((0, 9)),
                    groups=_log(rng, 4, 32), M=8 * _log(rng, 32, 256), N=8 * _log(rng, 32, 256),
                    skew=rng.choice((0.0, 0.5, 1.0)))
    g = rng.choice((32, 64, 128))
    case = dict(op=op, dtype=dtype, out=dtype if rng.random() < 0.7 else "f32", N=_log(rng, 256, 8192),
                K=g * _log(rng, 512 // g, 8192 // g), g=g, zeros=rng.random() < 0.5)
    if op == "qweight":
        return dict(case, M=_log(rng, 1, 2048))
    return dict(case, rows=_log(rng, 16, 2048), pad=rng.choice((0, 5)), groups=_log(rng, 4, 64),
                skew=rng.choice((0.0, 0.5, 1.0)))


def draw(rng):
    w = work(listed()[0])
    top = max(w["bytes"], w["flops"] / 50)
    while True:
        case = _draw(rng)
        w = work(case)
        if w["bytes"] < 1.5e9 and max(w["bytes"], w["flops"] / 50) <= top:
            return case


def work(case):
    op, e = case["op"], _SIZE[case["dtype"]]
    out = _SIZE[case["out"]]
    N = case["N"]
    if op == "grouped":
        rows, K = case["rows"], case["K"]
        hit = _touched(rows, case["groups"])
        b = rows * K * e + hit * K * N * e + rows * N * out + (hit * N * e if case["bias"] else 0)
        return {"bytes": b, "flops": 2 * rows * K * N}
    if op == "grouped_k":
        rows, M = case["rows"], case["M"]
        return {"bytes": rows * (M + N) * e + case["groups"] * M * N * out, "flops": 2 * rows * M * N}
    K, g = case["K"], case["g"]
    per = N * K / 2 + N * (K // g) * (e + (1 if case["zeros"] else 0))
    rows = case["M"] if op == "qweight" else case["rows"]
    hit = 1 if op == "qweight" else _touched(rows, case["groups"])
    return {"bytes": rows * K * e + hit * per + rows * N * out, "flops": 2 * rows * K * N}


def _touched(rows, groups):
    """Groups that get a row, about: rows fall on groups at random."""
    return groups * (1 - (1 - 1 / groups) ** rows)


def _rows_of_groups(case, gen):
    """Offsets of groups with unequal row counts (some may be empty), on the host."""
    w = torch.exp(case["skew"] * torch.randn(case["groups"], generator=gen))
    at = torch.multinomial(w, case["rows"], replacement=True, generator=gen)
    count = torch.bincount(at, minlength=case["groups"])
    return torch.cat([torch.zeros(1, dtype=torch.int64), count.cumsum(0)])


def prepare(case, seed):
    op, dt, out = case["op"], _DT[case["dtype"]], _DT[case["out"]]
    host = torch.Generator().manual_seed(seed)
    gen = torch.Generator(device="cuda").manual_seed(seed)

    def normal(*shape, std=1.0, dtype=dt):
        return torch.empty(shape, dtype=dtype, device="cuda").normal_(0.0, std, generator=gen)

    s = dict(case)
    if op != "qweight":
        off = _rows_of_groups(case, host)
        s["offsets"] = off.to(torch.int32).cuda()
        s["longest"] = int((off[1:] - off[:-1]).max())     # capacity of a group
        total = case["rows"] + case["pad"]
    if op == "grouped":
        G, K, N = case["groups"], case["K"], case["N"]
        s["A"] = normal(total, K)
        if case["order"] == "kn":
            s["B"] = normal(G, K, N, std=K ** -0.5)
        else:
            s["B"] = normal(G, N, K, std=K ** -0.5).transpose(1, 2)
        s["bias_v"] = normal(G, N, std=0.1) if case["bias"] else None
        s["C"] = torch.zeros(total, N, dtype=out, device="cuda")
    elif op == "grouped_k":
        s["A"] = normal(total, case["M"])
        s["B"] = normal(total, case["N"], std=0.05)
    else:
        N, K, g = case["N"], case["K"], case["g"]
        lead = (N,) if op == "qweight" else (case["groups"], N)
        q = torch.empty(lead + (K,), dtype=torch.float16, device="cuda").normal_(8.0, 3.0, generator=gen)
        q = q.round_().clamp_(0, 15).to(torch.uint8)
        s["Q"] = q[..., 0::2] | (q[..., 1::2] << 4)        # low four bits: even k
        u = torch.rand(lead + (K // g,), device="cuda", generator=gen)
        s["scales"] = ((0.5 + u) / (3.0 * K ** 0.5)).to(dt)
        s["zeros_v"] = (torch.randint(5, 12, lead + (K // g,), device="cuda", generator=gen, dtype=torch.uint8)
                        if case["zeros"] else None)
        rows = case["M"] if op == "qweight" else total
        s["A"] = normal(rows, K)
        s["C"] = torch.zeros(rows, N, dtype=out, device="cuda")
    return s


def run(s):
    return _own(s) if own else _plain(s)


def _own(s):
    import dense_gemm_10_amd as dg
    if s["op"] == "grouped":
        return dg.gemm_grouped(s["A"], s["B"], s["offsets"], s["C"], bias=s["bias_v"], act=s["act"])
    if s["op"] == "grouped_k":
        return dg.gemm_grouped_k(s["A"].t(), s["B"], s["offsets"], out_dtype=_DT[s["out"]])
    return dg.gemm_qweight(s["A"], s["Q"], s["scales"], s["zeros_v"], s["C"], group_size=s["g"],
                           offsets=s.get("offsets"))


def _act(v, act):
    if act == "gelu_erf":
        return 0.5 * v * (1.0 + torch.erf(v * (0.5 ** 0.5)))
    if act == "gelu_tanh":
        return 0.5 * v * (1.0 + torch.tanh((2.0 / math.pi) ** 0.5 * (v + 0.044715 * v * v * v)))
    return v


def _padded(x, off, cap):
    """Rows of each group of x in fp32, zero-filled to cap rows: (groups, cap, columns)."""
    at = off[:-1, None] + torch.arange(cap, device=x.device)
    inside = at < off[1:, None]
    return torch.where(inside[..., None], x[at.clamp(max=x.shape[0] - 1)].float(), 0.0)


def _back(padded, off, C):
    """The groups' rows in order; rows behind the last group stay as they are in C."""
    i = torch.arange(C.shape[0], device=C.device)
    e = torch.searchsorted(off[1:].contiguous(), i, right=True)
    inside = e < off.numel() - 1
    e = e.clamp(max=off.numel() - 2)
    at = (i - off[e]).clamp(min=0, max=padded.shape[1] - 1)
    return torch.where(inside[:, None], padded[e, at].to(C.dtype), C)


def _weights(s):
    q = torch.stack([s["Q"] & 15, s["Q"] >> 4], dim=-1).flatten(-2).float()
    q = q.unflatten(-1, (-1, s["g"]))
    zero = 8.0 if s["zeros_v"] is None else s["zeros_v"].float()[..., None]
    return ((q - zero) * s["scales"].float()[..., None]).flatten(-2)


def _plain(s):
    op = s["op"]
    if op == "qweight":
        return (s["A"].float() @ _weights(s).t()).to(s["C"].dtype)
    off = s["offsets"].long()
    a = _padded(s["A"], off, s["longest"])
    if op == "grouped_k":
        return torch.bmm(a.transpose(1, 2), _padded(s["B"], off, s["longest"])).to(_DT[s["out"]])
    if op == "grouped":
        v = torch.bmm(a, s["B"].float())
        if s["bias_v"] is not None:
            v = v + s["bias_v"].float()[:, None]
        return _back(_act(v, s["act"]), off, s["C"])
    return _back(torch.bmm(a, _weights(s).transpose(1, 2)), off, s["C"])


def exact(case, seed):
    """The definition, group by group, in fp64."""
    s = prepare(case, seed)
    op = s["op"]
    A = s["A"].double()
    off = [0, A.shape[0]] if op == "qweight" else s["offsets"].tolist()
    C = torch.zeros_like(s["C"], dtype=torch.float64) if op != "grouped_k" else []
    for e, (lo, hi) in enumerate(zip(off[:-1], off[1:])):
        if op == "grouped_k":
            C.append(A[lo:hi].t() @ s["B"][lo:hi].double())
            continue
        if op == "grouped":
            y = A[lo:hi] @ s["B"][e].double()
            if s["bias_v"] is not None:
                y += s["bias_v"][e].double()
            if s["act"] == "gelu_erf":
                y = y * torch.special.ndtr(y)
            elif s["act"] == "gelu_tanh":
                y = y / (1 + torch.exp(-2 * math.sqrt(2 / math.pi) * (y + 0.044715 * y ** 3)))
            C[lo:hi] = y
            continue
        pick = (lambda t: t) if op == "qweight" else (lambda t: t[e])
        q = pick(s["Q"])
        w = torch.empty(q.shape[0], s["K"], dtype=torch.float64, device=q.device)
        w[:, 0::2], w[:, 1::2] = (q % 16).double(), (q // 16).double()
        at = torch.arange(s["K"], device=q.device) // s["g"]
        w -= 8 if s["zeros_v"] is None else pick(s["zeros_v"]).double()[:, at]
        C[lo:hi] = A[lo:hi] @ (w * pick(s["scales"]).double()[:, at]).t()
    return torch.stack(C) if op == "grouped_k" else C
