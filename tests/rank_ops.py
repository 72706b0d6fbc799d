"""Shared helpers of the tests of a rank's forward and backward calls: buffers between guard bands, and the operators'
definitions in 64 bits."""
import math

import torch

U32 = torch.finfo(torch.float32).eps / 2  # a rounding to nearest of binary32, relative
GUARD, PATTERN = 4096, 0xA5
KINDS = ("layer", "rms")


def half_step(dtype):
    return torch.finfo(dtype).eps / 2


def least(dtype):
    """Half the least step between numbers of the type: a rounding of what is not normal is off by as much."""
    f = torch.finfo(dtype)
    return f.smallest_normal * f.eps / 2


class Guarded:
    """A matrix [rows, cols] whose rows lie `gap` elements apart, `skew` elements past a 256-byte boundary, in a buffer
    of a fixed byte pattern."""
    made = []

    def __init__(self, rows, cols, dtype, gap=0, skew=0, what=""):
        es = torch.empty(0, dtype=dtype).element_size()
        lead, self.what = GUARD // es + skew, what
        size = max(rows - 1, 0) * (cols + gap) + (cols if rows else 0)
        self.full = torch.empty((lead + size + GUARD // es) * es, dtype=torch.uint8, device="cuda")
        self.full.fill_(PATTERN)
        self.t = torch.as_strided(self.full.view(dtype), (rows, cols), (cols + gap, 1), lead)
        Guarded.made.append(self)

    def check(self):
        left = self.full.clone()
        inside = torch.as_strided(left.view(self.t.dtype), self.t.shape, self.t.stride(), self.t.storage_offset())
        inside.view(torch.uint8 if inside.element_size() == 1 else torch.int16
                    if inside.element_size() == 2 else torch.int32).fill_(0)
        mark = torch.full_like(self.full, PATTERN)
        marked = torch.as_strided(mark.view(self.t.dtype), self.t.shape, self.t.stride(), self.t.storage_offset())
        marked.view(torch.uint8 if marked.element_size() == 1 else torch.int16
                    if marked.element_size() == 2 else torch.int32).fill_(0)
        assert torch.equal(left, mark), f"{self.what}: written outside of its elements"


def check_guards():
    torch.cuda.synchronize()
    made, Guarded.made = Guarded.made, []
    for g in made:
        g.check()


def buffer(rows, cols, dtype, gap=0, skew=0, what=""):
    return Guarded(rows, cols, dtype, gap, skew, what).t


def filled(values, dtype, gap=0, skew=0, what=""):
    """A guarded matrix that holds `values` rounded to dtype."""
    t = buffer(*values.shape, dtype, gap, skew, what)
    t.copy_(values)
    return t


def bytes_buffer(n, what="workspace"):
    return Guarded(1, n, torch.uint8, what=what).t.view(-1)


def generator(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def normal(g, *shape):
    return torch.randn(*shape, generator=g, device="cuda")


# ---- checkpoints in 8 bits ---------------------------------------------------------------------------------------------

def e4m3_table():
    """The numbers of the codes 0 .. 126, ascending (127 is NaN; bit 7 is the sign)."""
    c = torch.arange(127, dtype=torch.float64)
    e, m = torch.div(c, 8, rounding_mode="floor"), c % 8
    return torch.where(e == 0, m * 2.0 ** -9, (8 + m) * torch.exp2(e - 10))


def keep(x):
    """(codes, scale bytes) of x by the definition, by trying: the least k, and the nearest code."""
    table = e4m3_table().to(x.device)
    largest = 8 if x.dtype == torch.float16 else 120
    rows, cols = x.shape
    groups = -(-cols // 32)
    v = torch.zeros(rows, groups * 32, dtype=torch.float64, device=x.device)
    v[:, :cols] = x.double()
    v = v.view(rows, groups, 32)
    fine = torch.isfinite(v)
    top = torch.where(fine, v.abs(), 0.0).amax(2)
    powers = torch.tensor([2.0 ** k for k in range(-100, 121)], dtype=torch.float64, device=x.device)
    k = torch.searchsorted(448.0 * powers, top) - 100
    scaled = torch.where(fine, v.abs(), 0.0) / powers[(k + 100)][:, :, None]
    above = torch.searchsorted(table, scaled).clamp(max=126)  # the first code that is not smaller
    below = (above - 1).clamp(min=0)
    up, down = table[above] - scaled, scaled - table[below]
    code = torch.where((up < down) | ((up == down) & (above % 2 == 0)), above, below)
    code = torch.where((k == largest)[:, :, None] & (table[code] > 240), 119, code)  # 119: 240
    code = torch.where(v.view(rows, groups, 32) < 0, code | 128, code)
    code = torch.where(torch.signbit(v) & (code < 128), code | 128, code)
    code = torch.where(fine, code, 127)
    return code.view(rows, -1)[:, :cols].to(torch.uint8), (k + 127).to(torch.uint8)


def numbers(codes, scales):
    """What a checkpoint stands for, in 64 bits."""
    table = torch.cat([e4m3_table(), torch.tensor([float("nan")], dtype=torch.float64)]).to(codes.device)
    v = table[(codes & 127).long()]
    v = torch.where(codes >= 128, -v, v)
    k = scales.double() - 127
    return v * torch.exp2(k.repeat_interleave(32, 1)[:, :codes.shape[1]])


def kept(zf, x, gap=0, skew=0):
    """A checkpoint of x by the definition, in buffers of its own."""
    codes, scales = keep(x)
    c = buffer(*codes.shape, torch.uint8, gap, skew, "codes")
    s = buffer(*scales.shape, torch.uint8, gap, skew, "scales")
    c.copy_(codes)
    s.copy_(scales)
    return zf.act8(c, s)


def blank(zf, rows, cols, gap=0, skew=0):
    return zf.act8(buffer(rows, cols, torch.uint8, gap, skew, "codes"),
                   buffer(rows, -(-cols // 32), torch.uint8, gap, skew, "scales"))


# ---- comparison --------------------------------------------------------------------------------------------------------

def assert_within(got, want, bound, what=""):
    """|got - want| <= bound, element by element; where want is not finite, got is the same kind.  A want that got's
    type cannot hold is an infinity there: rounding to nearest gives one from the largest number and half a step on
    (fp16: 65504 + 16 = 65520)."""
    f, exponent = torch.finfo(got.dtype), math.frexp(torch.finfo(got.dtype).max)[1]
    limit = f.max + f.eps * 2.0 ** (exponent - 2)
    got = got.double()
    bound = torch.as_tensor(bound, dtype=torch.float64, device=want.device).expand_as(want)
    over = torch.isinf(got) & (got.sign() == want.sign()) & (want.abs() + bound >= limit)
    got = torch.where(over, want, got)
    fine = torch.isfinite(want)
    assert bool((want.abs()[fine & ~over] - bound[fine & ~over] < limit).all()), \
        f"{what}: numbers where the type has none"
    assert torch.equal(fine, torch.isfinite(got)), f"{what}: other elements are infinite or NaN"
    bad = fine & ((got - want).abs() > bound)
    if bool(bad.any()):
        at = int(bad.flatten().nonzero()[0])
        raise AssertionError(f"{what}: {int(bad.sum())} of {bad.numel()} elements are off, the first at {at}: "
                             f"{float(got.flatten()[at])} for {float(want.flatten()[at])}, "
                             f"bound {float(bound.flatten()[at])}")


def rounded(want, error, dtype):
    """The bound of a result of `dtype` whose binary32 value is within `error` of `want`: one rounding more."""
    return error + (want.abs() + error) * half_step(dtype) + least(dtype)


def written(total, error, old, dtype, accumulate):
    """(value, bound) of a gradient that is stored, or added to `old` with a rounding of binary32."""
    if accumulate:
        total = total + old.double()
        error = error + (total.abs() + error) * U32
    return total, rounded(total, error, dtype)
