"""Measured cases of routed tokens and of the 8-bit products.

Four operators, all parts of a layer of experts or of one linear layer in 8 bits:

  dispatch     rows of x sorted by the group that each (token, choice) slot names, and the maps there and back;
               with "grad" the gradient of x from the rows' gradients
  combine      y[t] = sum_j w[t, j] z[place[t, j]]; with "grad" the gradients of z and w
  linear_i8    C = act(s[m] t[n] sum_k q[m, k] B[n, k] + bias[n]),  q[m] = rint(x[m] / s[m]),  s[m] = max |x[m]| / 127
  experts_i8   the same with one B, t and bias per group of rows

`own` false computes them with elementary torch operations, in fp32 but for the codes q, whose border cases need fp64;
`own` true calls the library.
"""
import math

import torch

own = False

_DT = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
_SIZE = {"bf16": 2, "f16": 2, "f32": 4}


def listed():
    return [
        # one generation step of 16 sequences: the smallest call
        dict(name="dispatch decode step", op="dispatch", dtype="bf16", tokens=16, top_k=2, groups=64, width=2048,
             index="i64", drop=0.0, skew=0.5, grad=False),
        # a training batch, there and its gradient
        dict(name="dispatch training batch", op="dispatch", dtype="bf16", tokens=8192, top_k=2, groups=16, width=4096,
             index="i64", drop=0.0, skew=0.5, grad=True),
        # a small fp32 layer of odd sizes, padding tokens that go to no expert
        dict(name="dispatch odd fp32", op="dispatch", dtype="f32", tokens=1001, top_k=3, groups=24, width=1037,
             index="i32", drop=0.1, skew=1.0, grad=True),
        # the way back of a generation step
        dict(name="combine decode step", op="combine", dtype="bf16", wtype="f32", tokens=16, top_k=2, groups=64,
             width=2048, drop=0.0, skew=0.5, grad=False),
        # the way back of a training batch with both gradients
        dict(name="combine training batch", op="combine", dtype="bf16", wtype="f32", tokens=8192, top_k=2, groups=16,
             width=4096, drop=0.0, skew=0.5, grad=True),
        # many choices per token, weights in the rows' type, padding tokens
        dict(name="combine eight choices fp16", op="combine", dtype="f16", wtype="f16", tokens=4095, top_k=8, groups=64,
             width=1000, drop=0.05, skew=0.5, grad=True),
        # one token through one square linear layer
        dict(name="8-bit one token 4096x4096", op="linear_i8", dtype="bf16", out="bf16", M=1, N=4096, K=4096,
             bias=False, act="none"),
        # a batch of sequences in generation through a wide layer
        dict(name="8-bit 13 tokens 16384x8192", op="linear_i8", dtype="f16", out="f16", M=13, N=16384, K=8192,
             bias=True, act="none"),
        # a prompt, bias and GELU fused
        dict(name="8-bit prompt 2048 tokens", op="linear_i8", dtype="bf16", out="bf16", M=2048, N=4096, K=4096,
             bias=True, act="gelu_tanh"),
        # odd sizes, rows that do not start on 16 bytes, fp32 out (logits)
        dict(name="8-bit odd 700 tokens 4097x1001", op="linear_i8", dtype="bf16", out="f32", M=700, N=4097, K=1001,
             bias=False, act="none"),
        # a generation step through 8-bit experts
        dict(name="8-bit experts decode step", op="experts_i8", dtype="bf16", out="bf16", rows=64, pad=0, groups=64,
             N=2048, K=2048, bias=False, act="none", skew=0.5),
        # a large batch through 8-bit experts: unequal groups, rows of no group behind the last
        dict(name="8-bit experts batch", op="experts_i8", dtype="bf16", out="bf16", rows=8192, pad=40, groups=16,
             N=4096, K=4096, bias=True, act="gelu_erf", skew=0.5),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _draw(rng):
    op = rng.choice(("dispatch", "combine", "linear_i8", "experts_i8"))
    dtype = rng.choice(("bf16", "f16", "f32"))
    if op in ("dispatch", "combine"):
        case = dict(op=op, dtype=dtype, tokens=_log(rng, 1, 16384), top_k=rng.choice((1, 2, 3, 4, 6, 8)),
                    groups=_log(rng, 2, 512), width=_log(rng, 256, 8192), drop=rng.choice((0.0, 0.0, 0.1)),
                    skew=rng.choice((0.0, 0.5, 1.0)), grad=rng.random() < 0.5)
        if rng.random() < 0.7:
            case["width"] = (case["width"] + 7) // 8 * 8
        if op == "dispatch":
            return dict(case, index=rng.choice(("i32", "i64")))
        return dict(case, wtype=rng.choice(("f32", dtype)))
    case = dict(op=op, dtype=dtype, out=rng.choice((dtype, dtype, "f32")), N=_log(rng, 256, 16384),
                K=_log(rng, 256, 8192), bias=rng.random() < 0.5, act=rng.choice(("none", "gelu_erf", "gelu_tanh")))
    if rng.random() < 0.7:
        case["K"] = (case["K"] + 15) // 16 * 16
    if op == "linear_i8":
        return dict(case, M=_log(rng, 1, 8192))
    return dict(case, rows=_log(rng, 16, 8192), pad=rng.choice((0, 7)), groups=_log(rng, 4, 64),
                skew=rng.choice((0.0, 0.5, 1.0)))


def draw(rng):
    top = max(_cost(c) for c in listed())
    while True:
        case = _draw(rng)
        if work(case)["bytes"] < 1e9 and _cost(case) <= top:
            return case


def _cost(case):
    w = work(case)
    return max(w["bytes"], w["flops"] / 50)


def work(case):
    op, e = case["op"], _SIZE[case["dtype"]]
    if op in ("dispatch", "combine"):
        T, S, D = case["tokens"], case["tokens"] * case["top_k"], case["width"]
        kept = S * (1 - case["drop"])
        if op == "dispatch":
            b = S * (8 if case["index"] == "i64" else 4) + T * D * e + kept * D * e + 8 * S + 4 * (case["groups"] + 1)
            return {"bytes": b + (kept * D * e + T * D * e if case["grad"] else 0),
                    "flops": kept * D if case["grad"] else 0}
        b = kept * D * e + S * (4 + _SIZE[case["wtype"]]) + T * D * e
        if case["grad"]:
            b += T * D * e + kept * D * e + S * _SIZE[case["wtype"]]
        return {"bytes": b, "flops": (5 if case["grad"] else 2) * kept * D}
    N, K = case["N"], case["K"]
    rows = case["M"] if op == "linear_i8" else case["rows"]
    hit = 1 if op == "linear_i8" else _touched(rows, case["groups"])
    per = N * K + 4 * N + (N * e if case["bias"] else 0)
    return {"bytes": rows * K * e + hit * per + rows * N * _SIZE[case["out"]], "flops": 2 * rows * N * K}


def _touched(rows, groups):
    """Groups that get a row, about: rows fall on groups at random."""
    return groups * (1 - (1 - 1 / groups) ** rows)


def _choices(case, host):
    """(tokens, top_k) groups, different ones within a token where there are enough; dropped tokens hold -1."""
    w = torch.exp(case["skew"] * torch.randn(case["groups"], generator=host))
    T, k = case["tokens"], case["top_k"]
    at = torch.multinomial(w.expand(T, -1), k, replacement=k > case["groups"], generator=host)
    at[torch.rand(T, generator=host) < case["drop"]] = -1
    return at


def _sorted_slots(at, groups):
    """place of every slot in the rows sorted by group, -1 for a dropped one, on the host."""
    flat = at.reshape(-1)
    key = torch.where(flat < 0, groups, flat)
    order = torch.sort(key, stable=True).indices
    place = torch.empty_like(order)
    place[order] = torch.arange(flat.numel())
    place[flat < 0] = -1
    return place.to(torch.int32).view_as(at)


def _rows_of_groups(case, gen):
    w = torch.exp(case["skew"] * torch.randn(case["groups"], generator=gen))
    at = torch.multinomial(w, case["rows"], replacement=True, generator=gen)
    count = torch.bincount(at, minlength=case["groups"])
    return torch.cat([torch.zeros(1, dtype=torch.int64), count.cumsum(0)])


def prepare(case, seed):
    op, dt = case["op"], _DT[case["dtype"]]
    host = torch.Generator().manual_seed(seed)
    gen = torch.Generator(device="cuda").manual_seed(seed)

    def normal(*shape, std=1.0, dtype=dt):
        return torch.empty(shape, dtype=dtype, device="cuda").normal_(0.0, std, generator=gen)

    s = dict(case)
    if op in ("dispatch", "combine"):
        T, k, D = case["tokens"], case["top_k"], case["width"]
        at = _choices(case, host)
        if op == "dispatch":
            s["at"] = at.to(torch.int32 if case["index"] == "i32" else torch.int64).cuda()
            s["x"] = normal(T, D)
            s["rows_out"] = torch.zeros(T * k, D, dtype=dt, device="cuda")
            if case["grad"]:
                s["drows"] = normal(T * k, D)
        else:
            s["place"] = _sorted_slots(at, case["groups"]).cuda()
            s["z"] = normal(T * k, D)
            s["w"] = torch.softmax(torch.randn(T, k, generator=host), -1).to(_DT[case["wtype"]]).cuda()
            if case["grad"]:
                s["dy"] = normal(T, D)
                s["dz"] = torch.zeros(T * k, D, dtype=dt, device="cuda")
        return s
    N, K = case["N"], case["K"]
    if op == "experts_i8":
        off = _rows_of_groups(case, host)
        s["offsets"] = off.to(torch.int32).cuda()
        s["longest"] = int((off[1:] - off[:-1]).max())     # capacity of a group
        rows, lead = case["rows"] + case["pad"], (case["groups"], N)
    else:
        rows, lead = case["M"], (N,)
    # activations have a few channels far larger than the others
    s["x"] = normal(rows, K)
    s["x"].mul_(torch.where(torch.rand(K, generator=host) < 0.01, 8.0, 1.0).to(dt).cuda())
    B = torch.empty(lead + (K,), dtype=torch.float16, device="cuda").normal_(0.0, 36.0, generator=gen)
    s["B"] = B.round_().clamp_(-127, 127).to(torch.int8)
    s["t"] = (0.5 + torch.rand(lead, device="cuda", generator=gen)) / (36.0 * K ** 0.5)
    s["bias_v"] = normal(*lead, std=0.1) if case["bias"] else None
    s["C"] = torch.zeros(rows, N, dtype=_DT[case["out"]], device="cuda")
    return s


def run(s):
    return _own(s) if own else _plain(s)


def _own(s):
    import dense_gemm_10_amd as dg
    op = s["op"]
    if op == "dispatch":
        rows, offsets, order, place = dg.dispatch_tokens(s["x"], s["at"], s["groups"], out=s["rows_out"])
        if s["grad"]:
            return rows, offsets, order, place, dg.combine_tokens(s["drows"], place)
        return rows, offsets, order, place
    if op == "combine":
        y = dg.combine_tokens(s["z"], s["place"], s["w"])
        if s["grad"]:
            return (y, *dg.combine_tokens_grad(s["dy"], s["z"], s["place"], s["w"], dz=s["dz"]))
        return y
    return dg.gemm_scaled(s["x"], s["B"], None, s["t"], s["C"], offsets=s.get("offsets"), bias=s["bias_v"], act=s["act"])


def _act(v, act):
    if act == "gelu_erf":
        return 0.5 * v * (1.0 + torch.erf(v * (0.5 ** 0.5)))
    if act == "gelu_tanh":
        return 0.5 * v * (1.0 + torch.tanh((2.0 / math.pi) ** 0.5 * (v + 0.044715 * v * v * v)))
    return v


def _picked(x, place):
    """Rows of x at every slot in fp32, zeros at the slots of no group."""
    return torch.where((place >= 0)[..., None], x[place.long().clamp(min=0)].float(), 0.0)


def _codes(x):
    """8-bit codes of every row (as floats) and the rows' scales."""
    top = x.abs().amax(-1, keepdim=True).double()
    q = torch.where(top > 0, x.double() * 127 / top, 0.0).round()
    return q.float(), (top / 127).float()


def _padded(x, off, cap):
    """Rows of each group of x, zero-filled to cap rows: (groups, cap, columns)."""
    at = off[:-1, None] + torch.arange(cap, device=x.device)
    inside = at < off[1:, None]
    return torch.where(inside[..., None], x[at.clamp(max=x.shape[0] - 1)], 0.0)


def _back(padded, off, C):
    """The groups' rows in order; rows behind the last group stay as they are in C."""
    i = torch.arange(C.shape[0], device=C.device)
    e = torch.searchsorted(off[1:].contiguous(), i, right=True)
    inside = e < off.numel() - 1
    e = e.clamp(max=off.numel() - 2)
    at = (i - off[e]).clamp(min=0, max=padded.shape[1] - 1)
    return torch.where(inside[:, None], padded[e, at].to(C.dtype), C)


def _plain(s):
    op = s["op"]
    if op == "dispatch":
        G, k = s["groups"], s["top_k"]
        flat = s["at"].reshape(-1).long()
        kept = (flat >= 0) & (flat < G)
        key = torch.where(kept, flat, G)
        order = torch.sort(key, stable=True).indices
        count = torch.zeros(G + 2, dtype=torch.int64, device=key.device).index_add_(0, key + 1, torch.ones_like(key))
        offsets = count[:G + 1].cumsum(0)
        i = torch.arange(flat.numel(), device=key.device)
        place = torch.empty_like(order)
        place[order] = i
        place = torch.where(kept, place, -1).view(s["at"].shape)
        order = torch.where(i < offsets[G], order, -1)
        rows = torch.where((order >= 0)[:, None], s["x"][order.clamp(min=0) // k], s["rows_out"])
        ints = tuple(v.to(torch.int32) for v in (offsets, order, place))
        if s["grad"]:
            return (rows, *ints, _picked(s["drows"], place).sum(1).to(s["x"].dtype))
        return (rows, *ints)
    if op == "combine":
        z, w = _picked(s["z"], s["place"]), s["w"].float()
        y = (z * w[..., None]).sum(1).to(s["z"].dtype)
        if not s["grad"]:
            return y
        dy, kept = s["dy"].float(), s["place"] >= 0
        dz = s["dz"].clone()
        dz[s["place"][kept].long()] = (dy[:, None] * w[..., None]).to(dz.dtype)[kept]
        return y, dz, (z * dy[:, None]).sum(-1).to(s["w"].dtype)
    q, scale = _codes(s["x"])
    if op == "linear_i8":
        v = (q @ s["B"].float().t()) * scale * s["t"]
        if s["bias_v"] is not None:
            v = v + s["bias_v"].float()
        return _act(v, s["act"]).to(s["C"].dtype)
    off = s["offsets"].long()
    v = torch.bmm(_padded(q, off, s["longest"]), s["B"].float().transpose(1, 2))
    v = v * _padded(scale, off, s["longest"]) * s["t"][:, None]
    if s["bias_v"] is not None:
        v = v + s["bias_v"].float()[:, None]
    return _back(_act(v, s["act"]), off, s["C"])


def exact(case, seed):
    """The definitions in fp64, group by group or choice by choice."""
    s = prepare(case, seed)
    op = s["op"]
    if op == "dispatch":
        T, k, G = s["tokens"], s["top_k"], s["groups"]
        lists = [[] for _ in range(G)]
        for slot, e in enumerate(s["at"].reshape(-1).tolist()):
            if 0 <= e < G:
                lists[e].append(slot)
        order = [slot for part in lists for slot in part]
        offsets = [0]
        for part in lists:
            offsets.append(offsets[-1] + len(part))
        place = [-1] * (T * k)
        for i, slot in enumerate(order):
            place[slot] = i
        ints = [torch.tensor(v, dtype=torch.int32, device="cuda")
                for v in (offsets, order + [-1] * (T * k - len(order)), place)]
        rows = s["rows_out"].double()
        rows[:len(order)] = s["x"].double()[ints[1][:len(order)].long() // k]
        out = (rows, ints[0], ints[1], ints[2].view(T, k))
        if not s["grad"]:
            return out
        dx = torch.zeros_like(s["x"], dtype=torch.float64)
        dx.index_add_(0, ints[1][:len(order)].long() // k, s["drows"][:len(order)].double())
        return (*out, dx)
    if op == "combine":
        y = torch.zeros(s["tokens"], s["width"], dtype=torch.float64, device="cuda")
        dz, dw = (s["dz"].double(), torch.zeros_like(s["w"], dtype=torch.float64)) if s["grad"] else (None, None)
        for j in range(s["top_k"]):
            t = (s["place"][:, j] >= 0).nonzero().flatten()
            at, w = s["place"][t, j].long(), s["w"][t, j].double()
            y[t] += w[:, None] * s["z"][at].double()
            if s["grad"]:
                dz[at] = w[:, None] * s["dy"][t].double()
                dw[t, j] = (s["z"][at].double() * s["dy"][t].double()).sum(1)
        return (y, dz, dw) if s["grad"] else y
    C = s["C"].double()
    off = [0, C.shape[0]] if op == "linear_i8" else s["offsets"].tolist()
    for e, (lo, hi) in enumerate(zip(off[:-1], off[1:])):
        if lo == hi:
            continue
        pick = (lambda t: t) if op == "linear_i8" else (lambda t: t[e])
        x = s["x"][lo:hi].double()
        top = x.abs().max(1, keepdim=True).values
        q = torch.round(127 * x / top.clamp(min=1e-300))
        y = (q @ pick(s["B"]).double().t()) * (top / 127) * pick(s["t"]).double()
        if s["bias_v"] is not None:
            y += pick(s["bias_v"]).double()
        if s["act"] == "gelu_erf":
            y = y * torch.special.ndtr(y)
        elif s["act"] == "gelu_tanh":
            y = y / (1 + torch.exp(-2 * math.sqrt(2 / math.pi) * (y + 0.044715 * y ** 3)))
        C[lo:hi] = y
    return C
