"""Plain forms of the token maps, sums and codes, on the CPU.

Tolerances, for one output:
  sum of k products in fp32, one fused multiply-add each: (k + 1) 2^-24 times
  the sum of absolute values (2^-23 below, for the rounded running sums);
  dot product of `width` terms in any order: (width + 8) 2^-23 times the sum
  of absolute values;
  output: half a step of the type, finfo(t).eps / 2, of the result with the
  errors above, and half the smallest subnormal.
Maps and codes are whole numbers and have to be equal.
"""
import torch

DT = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}


def maps(index, groups):
    """(offsets, order, place) of the definition."""
    flat = [int(v) for v in index.reshape(-1).tolist()]
    lists = [[] for _ in range(groups)]
    for s, e in enumerate(flat):
        if 0 <= e < groups:
            lists[e].append(s)
    offsets, order = [0], []
    for part in lists:
        order += part
        offsets.append(len(order))
    place = [-1] * len(flat)
    for i, s in enumerate(order):
        place[s] = i
    order += [-1] * (len(flat) - len(order))
    i32 = lambda v: torch.tensor(v, dtype=torch.int32)
    return i32(offsets), i32(order), i32(place).view(index.shape)


def random_index(tokens, top_k, groups, gen, drop=0.0, dtype=torch.int64):
    index = torch.randint(0, max(groups, 1), (tokens, top_k), generator=gen)
    index[torch.rand(tokens, top_k, generator=gen) < drop] = -1
    return index.to(dtype)


def rounded(ref, err, dtype):
    """Tolerance of ref, known up to err, once rounded to dtype."""
    info = torch.finfo(dtype)
    return err + info.eps / 2 * (ref.abs() + err) + info.smallest_normal * info.eps / 2


def combine64(z, place, w=None, y=None, beta=0.0):
    """(reference, sum of absolute values) in fp64."""
    tokens, top_k = place.shape
    out = torch.zeros(tokens, z.shape[1], dtype=torch.float64)
    mag = torch.zeros_like(out)
    for t in range(tokens):
        for j in range(top_k):
            p = int(place[t, j])
            if 0 <= p < z.shape[0]:
                v = z[p].double() * (1.0 if w is None else float(w[t, j]))
                out[t] += v
                mag[t] += v.abs()
    if y is not None:
        out += beta * y.double()
        mag += abs(beta) * y.double().abs()
    return out, mag


def codes64(x):
    """(codes, scales) of the definition."""
    x = x.double()
    top = x.abs().amax(1) if x.shape[1] else torch.zeros(x.shape[0], dtype=torch.float64)
    bad = ~torch.isfinite(x).all(1)
    q = torch.where((top > 0)[:, None], 127 * x / top[:, None], torch.zeros((), dtype=torch.float64)).round()
    q[bad] = 0
    scale = (top / 127).float()
    scale[bad] = float("nan")
    return q.to(torch.int8), scale


def same_bits(a, b):
    view = torch.int32 if a.element_size() == 4 else torch.int16 if a.element_size() == 2 else torch.int8
    return torch.equal(a.contiguous().view(view).cpu(), b.contiguous().view(view).cpu())
