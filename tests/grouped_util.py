"""Plain fp64 forms of the grouped and 4-bit-weight products, and the
tolerances of their tests.

Tolerances, for one output with K products:
  sum     fp32 accumulation in any order, each addition off by at most one
          unit in the last place (matrix cores may truncate): (K + 8) 2^-23
          times the sum of the products' absolute values;
  4 bit   the kernels may form sum a (16 + q) and sum a apart and subtract:
          the absolute values are then at most 31 |a| + 31 |a| per weight,
          times the scale, with K + K / group_size + 8 additions;
  act     GELU's slope is below 1.13 in absolute value; its own error is
          1.5e-7 |x| (the erf formula, Abramowitz and Stegun 7.1.26) plus four
          roundings of fp32, 2^-22 |y|, and the tanh form's argument error
          below 2^-20 |x|;
  output  half a step of the type, finfo(t).eps / 2, of the result with the
          errors above, and half the smallest subnormal.
"""
import torch

DT = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}


def act64(y, act):
    if act == "gelu_erf":
        return y * torch.special.ndtr(y)
    if act == "gelu_tanh":
        return y * torch.sigmoid(2 * (2 / torch.pi) ** 0.5 * (y + 0.044715 * y ** 3))
    return y


def groups_of(offsets, rows):
    """(start, end) of every group, as the header defines it."""
    out, top = [], 0
    off = [min(max(int(v), 0), rows) for v in offsets]
    top = off[0]
    for v in off[1:]:
        end = max(top, v)
        out.append((top, end))
        top = end
    return out


def finish(y, mag, err, out_dtype, *, alpha=1.0, beta=0.0, C=None, bias=None, act="none"):
    """(reference, tolerance) of act(alpha y + beta C + bias) in fp64; err is
    the error of y, mag its sum of absolute values (unused terms zero)."""
    v = alpha * y
    e = abs(alpha) * err + 2.0 ** -23 * abs(alpha) * y.abs()
    if C is not None and beta != 0.0:
        v = v + beta * C.double()
        e = e + 2.0 ** -23 * (beta * C.double()).abs()
    if bias is not None:
        v = v + bias.double()
        e = e + 2.0 ** -23 * (v.abs() + bias.double().abs())
    if act != "none":
        x = v
        v = act64(x, act)
        e = 1.13 * e + (1.5e-7 + 2.0 ** -20) * x.abs() + 2.0 ** -22 * v.abs()
    info = torch.finfo(out_dtype)
    half = info.eps / 2
    return v, e + half * (v.abs() + e) + info.smallest_normal * info.eps / 2


def sum_error(K, mag):
    return (K + 8) * 2.0 ** -23 * mag


def check(got, ref, tol, what=""):
    got = got.double().to(ref.device)
    assert got.shape == ref.shape
    bad = ~((got - ref).abs() <= tol)
    if bool(bad.any()):
        at = bad.nonzero()[:5].tolist()
        raise AssertionError(f"{what}: {int(bad.sum())} of {bad.numel()} outside the tolerance; first "
                             f"{[(i, float(got[tuple(i)]), float(ref[tuple(i)]), float(tol[tuple(i)])) for i in at]}")


def ints(gen, *shape, lo=-2, hi=2, dtype=torch.float32):
    """Small integers: every product and partial sum is exact."""
    return torch.randint(lo, hi + 1, shape, generator=gen).to(dtype)


def offsets_like(pattern, groups, rows, gen):
    """Offsets of one kind, as a list."""
    if pattern == "even":
        return [rows * e // groups for e in range(groups + 1)]
    if pattern == "random":
        cut = sorted(torch.randint(0, rows + 1, (groups - 1,), generator=gen).tolist())
        return [0] + cut + [rows]
    if pattern == "one":                    # one group has every row, the others none
        e = groups // 2
        return [0] * (e + 1) + [rows] * (groups - e)
    if pattern == "edges":                  # rows before the first and behind the last group
        lo, hi = min(3, rows), max(min(3, rows), rows - 5)
        inner = sorted(torch.randint(lo, hi + 1, (groups - 1,), generator=gen).tolist())
        return [lo] + inner + [hi]
    if pattern == "none":
        return [0] * (groups + 1)
    raise ValueError(pattern)
