"""Token operators on the GPU against plain 64-bit forms.

Tolerances, from the arithmetic:

Rotation. y = amplitude (a cos - b sin) in 32 bits, rounded once: half a step
of the output's type, plus amplitude (|a| + |b|) times
  the angle's rounding to 2^-32 of a turn and to 24 bits   pi 2^-25 + pi 2^-32
  sincospif, two ulp                                       2^-22
  the amplitude, the product and the sum                   3 * 2^-24
together below 6.2e-7 (ROT).

Attention. With W = sum p |v| / sum p per value, |out - exact| is at most half
a step of the output's type on |exact|, plus W times twice the relative error
of a weight p and of the sums:
  the score's sum of D products in 32 bits: D * 2^-23 * scale sum |q k|
  (a truncating accumulator errs by a step a product); a rotated query kept
  as two 16-bit values leaves 2^-16 of it
  exp2 and the remainder of p behind two 16-bit values: 2^-16 together, in
  fp16 2^-24 absolute as well (subnormal remainders)
  the sums over n tokens: (n / 16 + 64) * 2^-23
"""
import math

import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu

ROT = 6.2e-7
DT = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}


@pytest.fixture(scope="module")
def pkv():
    from paged_kv_cache_frame_b200 import build
    build.build()
    import paged_kv_cache_frame_b200 as m
    return m


def half_step(dtype):
    # the smallest normal's step below it (subnormal outputs)
    return torch.finfo(dtype).eps / 2, torch.finfo(dtype).tiny * torch.finfo(dtype).eps / 2


def gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def randn(shape, dtype, g):
    return torch.randn(shape, generator=g, device="cuda").to(dtype)


# ---------------------------------------------------------------- rotation
def turned(x, positions, rope, sign=1):
    """x [n, heads, d] rotated in 64 bits, angles reduced with an 80-bit product; and amplitude (|a| + |b|)."""
    x = x.detach().double().cpu().numpy()
    rot, amp = rope.rot_dim, rope.amplitude
    angle = np.asarray(positions.cpu().numpy(), dtype=np.longdouble)[:, None] * np.asarray(rope.inv_freq, np.longdouble)
    cos, sin = np.cos(angle).astype(np.float64)[:, None], sign * np.sin(angle).astype(np.float64)[:, None]
    y, w = x.copy(), np.zeros_like(x)
    i = (slice(0, rot // 2), slice(rot // 2, rot)) if rope.layout == "half" else (slice(0, rot, 2), slice(1, rot, 2))
    a, b = x[..., i[0]], x[..., i[1]]
    y[..., i[0]] = amp * (a * cos - b * sin)
    y[..., i[1]] = amp * (b * cos + a * sin)
    w[..., i[0]] = w[..., i[1]] = amp * (np.abs(a) + np.abs(b))
    return y, w


def assert_turned(got, x, positions, rope, sign=1):
    y, w = turned(x, positions, rope, sign)
    eps, tiny = half_step(got.dtype)
    err = np.abs(got.detach().double().cpu().numpy() - y)
    tol = np.where(w > 0, eps * (np.abs(y) + ROT * w) + ROT * w + tiny, 0)   # what is not rotated keeps its bits
    assert (err <= tol).all(), f"worst {np.max(err - tol):.3e}"


def ropes(pkv, rot, layout):
    return {
        "none": pkv.Rope(rot, layout=layout),
        "linear": pkv.Rope(rot, layout=layout, scaling="linear", factor=3.0),
        "ntk": pkv.Rope(rot, layout=layout, scaling="ntk", factor=8.0, base=500000.0),
        "yarn": pkv.Rope(rot, layout=layout, scaling="yarn", factor=16.0, original_context=2048),
    }


@pytest.mark.parametrize("dtype", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("layout", ["half", "interleaved"])
@pytest.mark.parametrize("n,h,d,rot,scaling", [
    (1, 1, 64, 64, "none"), (33, 5, 128, 128, "yarn"), (7, 40, 128, 64, "linear"), (257, 3, 80, 80, "ntk"),
    (19, 2, 96, 34, "yarn"), (5, 17, 256, 256, "none"), (3, 1, 66, 2, "none"), (64, 7, 512, 250, "linear"),
    (4001, 9, 64, 48, "ntk"), (2, 300, 2, 2, "none")])
def test_rotate(pkv, dtype, layout, n, h, d, rot, scaling):
    g = gen(n * 7 + d)
    rope = ropes(pkv, rot, layout)[scaling]
    x = randn((n, h, d), DT[dtype], g)
    pos = torch.randint(-10, 200000, (n,), generator=g, device="cuda", dtype=torch.int32)
    keep = x.clone()
    assert_turned(rope.rotate(x, pos), keep, pos, rope)
    assert_turned(rope.rotate(x, pos, inverse=True), keep, pos, rope, -1)
    assert torch.equal(x, keep)
    assert rope.rotate(x, pos, out=x) is x
    assert_turned(x, keep, pos, rope)


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_rotate_far_positions(pkv, dtype):
    pos = torch.tensor([0, 1, -1, 2**24 + 1, 10**6 + 7, 2**31 - 1, -2**31, -123456789], dtype=torch.int32, device="cuda")
    x = randn((8, 3, 128), DT[dtype], gen(3))
    for rope in (*ropes(pkv, 128, "half").values(), pkv.Rope(6, inv_freq=[64.0, -0.3, 0.0])):
        assert_turned(rope.rotate(x, pos), x, pos, rope)
    with pytest.raises(pkv.KVError):                # its angles could not be told apart at far positions
        pkv.Rope(6, inv_freq=[1e6, -0.3, 0.0])


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("layout", ["half", "interleaved"])
def test_rotate_strides_and_alignment(pkv, dtype, layout):
    """Slices of a fused projection, heads outside of tokens, rows off the 16-byte grid, and what lies between them."""
    g, rope = gen(4), pkv.Rope(48, layout=layout)
    pos = torch.arange(11, device="cuda", dtype=torch.int32)
    fused = randn((11, 6 * 64 + 3), DT[dtype], g)
    for x in (fused[:, :384].view(11, 6, 64)[:, 1:4], fused[:, 3:].view(11, 6, 64),
              randn((5, 11, 64), DT[dtype], g).transpose(0, 1), randn((1, 1, 64), DT[dtype], g).expand(11, 2, 64)):
        assert_turned(rope.rotate(x, pos), x, pos, rope)
    hold = torch.full((11, 9, 70), 7.0, device="cuda", dtype=DT[dtype])
    x = randn((11, 4, 64), DT[dtype], g)
    rope.rotate(x, pos, out=hold[:, 2:6, 3:67])
    assert_turned(hold[:, 2:6, 3:67], x, pos, rope)
    hold[:, 2:6, 3:67] = 7.0
    assert (hold == 7).all()


def test_rotate_empty(pkv):
    rope = pkv.Rope(64)
    for shape in ((0, 2, 64), (3, 0, 64)):
        pos = torch.zeros(shape[0], dtype=torch.int32, device="cuda")
        assert rope.rotate(torch.zeros(shape, device="cuda"), pos).shape == shape


@pytest.mark.parametrize("layout,rot,dtype", [("half", 64, "fp32"), ("interleaved", 20, "fp32"), ("half", 12, "bf16")])
def test_rotate_gradient(pkv, layout, rot, dtype):
    g = gen(5)
    rope = pkv.Rope(rot, layout=layout, scaling="yarn", factor=4.0, original_context=512)
    pos = torch.randint(0, 5000, (13,), generator=g, device="cuda", dtype=torch.int32)
    x = randn((13, 3, 64), DT[dtype], g).requires_grad_()
    dy = randn((13, 3, 64), DT[dtype], g)
    y = rope.rotate(x, pos)
    dx, = torch.autograd.grad(y, x, dy)
    assert_turned(y, x, pos, rope)
    assert_turned(dx, dy, pos, rope, -1)            # the formula's
    if dtype == "fp32":                             # differences: the rotation is linear, so a whole step will do
        for i in range(0, 64, 7):
            e = torch.zeros_like(x)
            e[:, :, i] = 1
            with torch.no_grad():
                d = ((rope.rotate(x + e, pos) - rope.rotate(x - e, pos)).double() / 2 * dy.double()).sum(-1)
            # |x| <= 6 and |dy| <= 6: three roundings of 2^-24 on values below 12, over at most two terms
            assert (d - dx[:, :, i].double()).abs().max() < 2 * 6 * 4 * 12 * 2**-24
    # a broadcast gradient (stride 0), a transposed one, and the gradient's gradient
    dx, = torch.autograd.grad(rope.rotate(x, pos).sum(), x)
    assert_turned(dx, torch.ones_like(x), pos, rope, -1)
    dt = randn((13, 64, 3), DT[dtype], g).transpose(1, 2)
    dx, = torch.autograd.grad(rope.rotate(x, pos), x, dt)
    assert_turned(dx, dt, pos, rope, -1)
    v = dy.clone().requires_grad_()
    dx, = torch.autograd.grad(rope.rotate(x, pos), x, v, create_graph=True)
    dv, = torch.autograd.grad(dx, v, dt)
    assert_turned(dv, dt, pos, rope)


def test_rotate_gradient_outlives_the_handle(pkv):
    pos = torch.arange(9, device="cuda", dtype=torch.int32)
    x = torch.randn(9, 2, 64, device="cuda", requires_grad=True)
    rope = pkv.Rope(64, base=77.0)
    y = rope.rotate(x, pos)
    del rope
    dy = torch.randn_like(y)
    dx, = torch.autograd.grad(y, x, dy)
    assert_turned(dx, dy, pos, pkv.Rope(64, base=77.0), -1)


def test_rotate_gradient_sees_changed_positions(pkv):
    pos = torch.arange(4, device="cuda", dtype=torch.int32)
    x = torch.randn(4, 2, 64, device="cuda", requires_grad=True)
    y = pkv.Rope(64).rotate(x, pos)
    pos += 1
    with pytest.raises(RuntimeError):
        y.sum().backward()


# ---------------------------------------------------------------- paged sequences
class Batch:
    """Sequences with pages in random order, rows past each length poisoned, and entries past the last page out of range."""

    def __init__(self, pkv, lens, hkv, d, page, dtype="bf16", seed=0, width=None, first_page=0, poison=True):
        self.g = gen(seed)
        self.lens, self.page, self.hkv, self.d, self.dtype = list(lens), page, hkv, d, DT[dtype]
        pages = [-(-n // page) for n in lens]
        width = width or max(max(pages, default=1), 1)
        count = first_page + sum(pages) + 2
        self.pool = torch.empty((count, 2, page, hkv, d), dtype=self.dtype, device="cuda")
        self.pool[first_page:] = math.nan if poison else 0
        order = (torch.randperm(count - first_page, generator=self.g, device="cuda") + first_page).tolist()
        self.rows, at = [], 0
        for n in pages:
            self.rows.append(order[at:at + n])
            at += n
        bad = [-1, count, 2**31 - 1, -2**31]
        table = [r + [bad[i % 4] for i in range(width - len(r))] for r in self.rows]
        self.tables = torch.tensor(table, dtype=torch.int32, device="cuda").view(len(lens), width)
        self.len_t = torch.tensor(self.lens, dtype=torch.int32, device="cuda")
        for s, n in enumerate(lens):
            p, r = self.where(s, torch.arange(n, device="cuda"))
            self.pool[p, 0, r] = randn((n, hkv, d), self.dtype, self.g)
            self.pool[p, 1, r] = randn((n, hkv, d), self.dtype, self.g)
        self.cache = pkv.PagedTokens(self.pool, self.tables, self.len_t)

    def where(self, s, j):
        return torch.tensor(self.rows[s] + [0], device="cuda")[j // self.page], j % self.page

    def kv(self, s, n):
        p, r = self.where(s, torch.arange(n, device="cuda"))
        return self.pool[p, 0, r].double(), self.pool[p, 1, r].double()


def attended(k, v, q, scale, window):
    """Exact output, W and the score's sum |q k| bound of one sequence: k, v [n, hkv, d], q [hq, d], all 64 bits."""
    n, hkv, d = k.shape
    g = q.shape[0] // hkv
    a = max(0, n - window) if window else 0
    k, v = k[a:].permute(1, 0, 2), v[a:].permute(1, 0, 2)
    q = q.view(hkv, g, d)
    s = scale * q @ k.transpose(1, 2)
    p = (s - s.amax(-1, keepdim=True)).exp()
    l = p.sum(-1, keepdim=True)
    most = abs(scale) * (q.abs() @ k.abs().transpose(1, 2)).amax(-1, keepdim=True)
    return (p @ v / l).view(-1, d), (p @ v.abs() / l).view(-1, d), (v.abs().sum(1, keepdim=True) / l).view(-1, d), \
        most.expand(hkv, g, d).reshape(-1, d), n - a


def assert_attended(out, b, q, scale=None, window=0, extra=0.0, kv=None):
    scale = b.d ** -0.5 if scale is None else scale
    eps, tiny = half_step(out.dtype)
    for s, n in enumerate(b.lens):
        if n == 0:
            assert (out[s] == 0).all()
            continue
        k, v = kv[s] if kv else b.kv(s, n)
        want, w, flat, most, seen = attended(k, v, q[s].double(), scale, window)
        rel = most * (b.d * 2**-23 + extra) + 2**-16 + (seen / 16 + 64) * 2**-23
        tol = eps * want.abs() + tiny + 2 * rel * w * (1 + eps) + (flat * 2**-24 if out.dtype == torch.float16 else 0)
        err = (out[s].double() - want).abs()
        assert bool((err <= tol).all()), f"sequence {s}: worst {float((err - tol).max()):.3e} of {float(tol.max()):.3e}"


DECODE = [
    # lens, kv heads, group, head_dim, page, dtype, window
    ([1], 1, 1, 64, 1, "bf16", 0), ([2], 2, 3, 128, 7, "fp16", 0), ([16, 17, 15], 2, 8, 128, 16, "bf16", 0),
    ([31, 32, 33, 0, 1], 4, 2, 64, 5, "fp16", 0), ([63, 64, 65, 127, 128, 129], 1, 9, 128, 64, "bf16", 0),
    ([300], 16, 1, 64, 256, "bf16", 0), ([999, 1000, 1998], 3, 16, 64, 999, "fp16", 0),
    ([0, 0, 5, 0], 2, 17, 128, 3, "bf16", 0), ([20000], 1, 4, 128, 64, "fp16", 0), ([20352], 16, 1, 64, 256, "bf16", 0),
    ([1000, 10, 0, 700], 2, 5, 128, 33, "bf16", 100), ([513, 100, 99, 101], 4, 7, 64, 17, "fp16", 100),
    ([4000, 1], 8, 4, 128, 128, "bf16", 1), ([5000] * 3, 1, 40, 64, 16, "bf16", 4097)]


@pytest.mark.parametrize("lens,hkv,g,d,page,dtype,window", DECODE, ids=lambda x: str(x)[:24])
def test_decode(pkv, lens, hkv, g, d, page, dtype, window):
    b = Batch(pkv, lens, hkv, d, page, dtype, seed=len(lens) + page)
    q = randn((len(lens), hkv * g, d), b.dtype, b.g)
    out = b.cache.decode(q, window=window)
    b.cache.check_device()
    assert_attended(out, b, q, window=window)
    assert torch.equal(out, b.cache.decode(q, window=window))   # no result depends on timing


@pytest.mark.parametrize("d,dtype", [(64, "bf16"), (128, "fp16")])
def test_decode_many_sequences(pkv, d, dtype):
    """More sequences than a block has threads and than the grid has CTAs, most of them short."""
    rng = np.random.default_rng(1)
    lens = [int(x) for x in rng.integers(0, 40, 700)]
    lens[350] = 9000
    b = Batch(pkv, lens, 2, d, 13, dtype, seed=2)
    q = randn((700, 4, d), b.dtype, b.g)
    assert_attended(b.cache.decode(q), b, q)
    b.cache.check_device()


@pytest.mark.parametrize("fused", [False, True])
def test_as_many_sequences_as_a_call_takes_and_coarse_tiles(pkv, fused):
    """16384 sequences whose tables could name 2^24 tokens each: the split counts in coarser tiles. The sequences share
    four pages (none that a new token goes to, but for one's own last)."""
    n, page, width, g = 16384, 65536, 256, gen(26)
    pool = randn((5, 2, page, 1, 64), torch.bfloat16, g)
    lens = torch.ones(n, dtype=torch.int32)
    some = {5: 0, 100: 300, 9000: 257, 9001: 0, 16383: 40000}
    for s, x in some.items():
        lens[s] = x
    tables = torch.full((n, width), -1, dtype=torch.int32)
    tables[:, 0] = torch.arange(n) % 4
    if fused:                                       # only one sequence appends: the others are unused
        tables[16383, 0] = 4
        lens[:16383] = 0
    cache = pkv.PagedTokens(pool, tables.cuda(), lens.cuda())
    q = randn((n, 2, 64), torch.bfloat16, g)
    if fused:
        k, v = randn((n, 1, 64), torch.bfloat16, g), randn((n, 1, 64), torch.bfloat16, g)
        out = cache.decode_append(k, v, q)
        assert torch.equal(pool[4, 0, 39999], k[16383]) and torch.equal(pool[4, 1, 39999], v[16383])
    else:
        out = cache.decode(q)
    cache.check_device()
    b = Batch.__new__(Batch)
    b.d = 64
    for s in some:
        b.lens = [int(lens[s])]
        p = int(tables[s, 0])
        kv = pool[p, :, :b.lens[0]].double()
        assert_attended(out[s:s + 1], b, q[s:s + 1], kv=[(kv[0], kv[1])])
    one = torch.ones(n, dtype=torch.bool)
    one[list(some)] = False
    if fused:
        assert (out[one.cuda()] == 0).all()
    else:                                           # one token: its value, to the bit
        want = pool[tables[:, 0].cuda().long(), 1, 0].expand(n, 2, 64)
        assert torch.equal(out[one.cuda()], want[one.cuda()])


@pytest.mark.parametrize("hkv,g", [(300, 1), (149, 2), (148, 1), (3, 1600)])
def test_more_heads_than_the_gpu_has_room_for(pkv, hkv, g):
    """Units that fill the GPU alone: a CTA each, and nothing to join."""
    b = Batch(pkv, [700, 0, 33], hkv, 64, 40, "fp16", seed=27)
    q = randn((3, hkv * g, 64), b.dtype, b.g)
    assert_attended(b.cache.decode(q), b, q)
    k, v = randn((3, hkv, 64), b.dtype, b.g), randn((3, hkv, 64), b.dtype, b.g)
    before = b.pool.clone()
    out = b.cache.decode_append(k, v, q)
    assert_appended(b, before, [1, 1, 1], k, v, None)
    assert_attended(out, b, q)
    b.cache.check_device()


def test_decode_nothing(pkv):
    b = Batch(pkv, [0, 0], 2, 64, 16, width=2)
    out = torch.full((2, 4, 64), 3.0, dtype=torch.bfloat16, device="cuda")
    b.cache.decode(randn((2, 4, 64), b.dtype, b.g), out=out)
    assert (out == 0).all()
    empty = pkv.PagedTokens(b.pool, b.tables[:0], b.len_t[:0])
    assert empty.decode(out[:0]).shape == (0, 4, 64)
    b.cache.check_device()


@pytest.mark.parametrize("scale", [1.0, -0.5, 8.0, 1e-4])
def test_decode_scales(pkv, scale):
    """Peaked and flat weights: a scale of 8 leaves one token, and running maxima that grow late."""
    b = Batch(pkv, [700, 3], 2, 128, 50, "bf16", seed=8)
    q = randn((2, 6, 128), b.dtype, b.g)
    p, r = b.where(0, torch.tensor([690], device="cuda"))
    b.pool[p, 0, r] = (b.pool[p, 0, r].float() * 3).to(b.dtype)
    assert_attended(b.cache.decode(q, scale=scale), b, q, scale=scale)


def test_decode_strides(pkv):
    b = Batch(pkv, [100, 200, 50], 4, 64, 32, seed=9)
    fused = randn((3, 12 * 64 + 8), b.dtype, b.g)
    q = fused[:, 8:].view(3, 12, 64)[:, 2:10]
    assert_attended(b.cache.decode(q), b, q)
    q = randn((8, 3, 64), b.dtype, b.g).transpose(0, 1)
    assert_attended(b.cache.decode(q), b, q)
    with pytest.raises(pkv.KVError):
        b.cache.decode(fused[:, 4:772].view(3, 12, 64))     # rows off the 16-byte grid
    wide = torch.zeros((3, 40), dtype=torch.int32, device="cuda")
    wide[:, 5:5 + b.tables.shape[1]] = b.tables
    c = pkv.PagedTokens(b.pool, wide[:, 5:5 + b.tables.shape[1]], b.len_t)
    assert torch.equal(c.decode(q), b.cache.decode(q))


def test_decode_infinite_values_outside(pkv):
    """Infinities and NaN past the length, before the window and in pages of no sequence change nothing."""
    b = Batch(pkv, [500], 2, 128, 64, "fp16", seed=10)
    q = randn((1, 4, 128), b.dtype, b.g)
    want = b.cache.decode(q, window=77)
    p, r = b.where(0, torch.arange(423, device="cuda"))
    b.pool[p, :, r] = math.inf
    assert torch.equal(b.cache.decode(q, window=77), want)
    assert_attended(want, b, q, window=77)


def test_decode_bad_pages_are_left_out_and_reported(pkv):
    b = Batch(pkv, [400, 100, 64], 2, 64, 32, seed=11)
    q = randn((3, 4, 64), b.dtype, b.g)
    for bad in (-1, b.pool.shape[0], 2**31 - 1):
        t = b.tables.clone()
        t[0, 3] = bad
        t[2, 0] = t[2, 1] = bad
        c = pkv.PagedTokens(b.pool, t, b.len_t)
        out = c.decode(q)
        with pytest.raises(pkv.KVError) as e:
            c.check_device()
        assert e.value.name == "DEVICE_CHECK"
        c.check_device()                                    # cleared
        k, v = b.kv(0, 400)
        keep = torch.ones(400, dtype=torch.bool, device="cuda")
        keep[96:128] = False
        assert (out[2] == 0).all()
        some = Batch.__new__(Batch)
        some.lens, some.d = [368, 100], 64
        assert_attended(out[:2], some, q[:2], kv=[(k[keep], v[keep]), b.kv(1, 100)])


def test_decode_lengths_out_of_range_are_held_and_reported(pkv):
    b = Batch(pkv, [64, 40], 1, 64, 16, seed=12)
    q = randn((2, 2, 64), b.dtype, b.g)
    b.len_t.copy_(torch.tensor([10**9, -3], dtype=torch.int32))
    out = b.cache.decode(q)
    with pytest.raises(pkv.KVError):
        b.cache.check_device()
    b.lens = [64, 0]
    assert_attended(out, b, q)


def test_offsets_past_32_bits(pkv):
    """A pool of 11 GB, the sequences' pages behind element 2^32."""
    page, hkv, d = 256, 16, 128
    first = (2**32) // (2 * page * hkv * d) + 1
    b = Batch(pkv, [700, 300], hkv, d, page, seed=13, first_page=first)
    assert b.pool[first:].storage_offset() > 2**32
    q = randn((2, hkv, d), b.dtype, b.g)
    assert_attended(b.cache.decode(q), b, q)
    k, v = (randn((2, hkv, d), b.dtype, b.g) for _ in range(2))
    b.cache.append(k, v)
    p, r = b.where(0, torch.tensor([699], device="cuda"))
    assert torch.equal(b.pool[p, 0, r][0], k[0]) and torch.equal(b.pool[p, 1, r][0], v[0])
    out = b.cache.decode_append(v, k, q)
    assert torch.equal(b.pool[p, 0, r][0], v[0]) and torch.equal(b.pool[p, 1, r][0], k[0])
    assert_attended(out, b, q)


# ---------------------------------------------------------------- appending
def assert_appended(b, before, new, k, v, rope, pos=None):
    """The pool holds the new tokens, keys rotated, and is otherwise `before`, bit for bit."""
    want, at = before, 0
    bits = (lambda x: x.view(torch.int16))
    for s, m in enumerate(new):
        n = b.lens[s]
        if n:
            j = torch.arange(n - m, n, device="cuda")
            p, r = b.where(s, j)
            ks = k[at:at + m]
            if rope is None:
                assert torch.equal(b.pool[p, 0, r], ks)
            else:
                assert_turned(b.pool[p, 0, r], ks, j if pos is None else pos[at:at + m], rope)
            assert torch.equal(bits(b.pool[p, 1, r]), bits(v[at:at + m]))
            want[p, :, r] = b.pool[p, :, r]
        at += m
    assert torch.equal(bits(b.pool), bits(want))


@pytest.mark.parametrize("dtype,d", [("bf16", 64), ("fp16", 128)])
@pytest.mark.parametrize("layout,rot", [("half", 64), ("half", 20), ("interleaved", 50), (None, 0)])
@pytest.mark.parametrize("lens,new,page,hkv,pad", [
    ([1], [1], 1, 1, 0), ([5, 0, 9], [1, 1, 1], 4, 3, 0), ([40, 64, 0, 7, 300], [40, 1, 0, 0, 77], 16, 2, 5),
    ([2500, 130], [2500, 1], 999, 16, 0), ([30] * 70, [3] * 70, 7, 8, 1)], ids=lambda x: str(x)[:20])
def test_append(pkv, dtype, d, layout, rot, lens, new, page, hkv, pad):
    b = Batch(pkv, lens, hkv, d, page, dtype, seed=page + rot)
    rope = pkv.Rope(rot, layout=layout) if layout else None
    n = sum(new) + pad
    k, v = randn((n, hkv, d), b.dtype, b.g), randn((n, hkv, d), b.dtype, b.g)
    cu = torch.tensor(np.cumsum([0] + new), dtype=torch.int32, device="cuda")
    before = b.pool.clone()
    b.cache.append(k, v, cu_new=cu, rope=rope)
    b.cache.check_device()
    assert_appended(b, before.clone(), new, k, v, rope)
    if new == [1] * len(new):                       # the same as one token each
        got = b.pool.clone()
        b.pool.copy_(before)
        b.cache.append(k, v, rope=rope)
        assert torch.equal(got.view(torch.int16), b.pool.view(torch.int16))
    if rope:
        pos = torch.randint(0, 100000, (n,), generator=b.g, device="cuda", dtype=torch.int32)
        b.pool.copy_(before)
        b.cache.append(k, v, cu_new=cu, rope=rope, positions=pos)
        assert_appended(b, before, new, k, v, rope, pos)


def test_append_strides(pkv):
    b = Batch(pkv, [3, 4], 2, 64, 8, seed=14)
    fused = randn((2, 8 * 64), b.dtype, b.g).view(2, 8, 64)
    before = b.pool.clone()
    rope = pkv.Rope(64)
    b.cache.append(fused[:, 4:6], fused[:, 6:], rope=rope)
    assert_appended(b, before, [1, 1], fused[:, 4:6], fused[:, 6:], rope)
    with pytest.raises(pkv.KVError):
        k = randn((2, 2 * 64 + 4), b.dtype, b.g)[:, 4:].view(2, 2, 64)
        b.cache.append(k, k)


def test_append_out_of_range_is_left_out_and_reported(pkv):
    b = Batch(pkv, [20, 20, 20], 2, 64, 8, seed=15)
    before = b.pool.clone().view(torch.int16)
    k = randn((9, 2, 64), b.dtype, b.g)
    t = b.tables.clone()
    t[0, 2] = b.pool.shape[0]
    c = pkv.PagedTokens(b.pool, t, b.len_t)
    for cu in ([0, 2, 2, 2], [0, 0, 21, 21], [3, 3, 2, 9], [9, 8, 7, 6], [-5, -5, -5, -5], [5, 5, 5, 5]):
        n = 25 if max(cu) > 9 else 9
        kk = randn((n, 2, 64), b.dtype, b.g)
        cu_t = torch.tensor(cu, dtype=torch.int32, device="cuda")
        b.pool.view(torch.int16).copy_(before)
        c.append(kk, kk, cu_new=cu_t)
        if cu == [-5, -5, -5, -5]:
            c.check_device()                        # every token lies behind the last sequence
        else:
            with pytest.raises(pkv.KVError):
                c.check_device()
        if cu in ([0, 2, 2, 2], [-5, -5, -5, -5]):
            assert torch.equal(b.pool.view(torch.int16), before)


# ---------------------------------------------------------------- the decode step
STEP = [
    ([1], 1, 1, 64, 1, "bf16", 0, "half", 64), ([40, 0, 1, 64, 65], 2, 4, 128, 16, "fp16", 0, "half", 128),
    ([513, 1000], 8, 2, 128, 256, "bf16", 0, "interleaved", 64), ([33, 300, 0, 31, 32], 3, 7, 64, 9, "bf16", 50, "half", 20),
    ([9000], 2, 17, 64, 64, "fp16", 0, None, 0), ([128] * 20, 1, 16, 128, 128, "bf16", 1, "interleaved", 126),
    ([5, 700], 4, 33, 128, 999, "bf16", 0, "half", 96)]


@pytest.mark.parametrize("lens,hkv,g,d,page,dtype,window,layout,rot", STEP, ids=lambda x: str(x)[:20])
def test_decode_append(pkv, lens, hkv, g, d, page, dtype, window, layout, rot):
    b = Batch(pkv, lens, hkv, d, page, dtype, seed=16 + d)
    rope = pkv.Rope(rot, layout=layout, scaling="yarn", factor=4.0, original_context=64) if layout else None
    s = len(lens)
    q = randn((s, hkv * g, d), b.dtype, b.g)
    k, v = randn((s, hkv, d), b.dtype, b.g), randn((s, hkv, d), b.dtype, b.g)
    for n, row in zip(lens, range(s)):              # the slot's old content must not count
        if n:
            p, r = b.where(row, torch.tensor([n - 1], device="cuda"))
            b.pool[p, :, r] = math.nan
    before = b.pool.clone()
    for pos in (None, torch.randint(-9, 70000, (s,), generator=b.g, device="cuda", dtype=torch.int32)):
        b.pool.copy_(before)
        out = b.cache.decode_append(k, v, q, rope=rope, positions=pos, window=window)
        b.cache.check_device()
        assert_appended(b, before.clone(), [min(1, n) for n in lens] if 0 not in lens else [1] * s, k, v, rope, pos)
        at = b.len_t.long() - 1 if pos is None else pos
        exact_q = torch.tensor(turned(q, at, rope)[0], device="cuda") if rope else q
        assert_attended(out, b, exact_q, window=window, extra=2**-16 + ROT)
        # the three calls apart: the pool bit for bit, the output but for the query's rounding
        got = b.pool.clone()
        b.pool.copy_(before)
        b.cache.append(k, v, rope=rope, positions=pos)
        assert torch.equal(got.view(torch.int16), b.pool.view(torch.int16))
        if rope is None:
            assert torch.equal(b.cache.decode(q, window=window), out)


def test_decode_append_bad_page(pkv):
    b = Batch(pkv, [17, 40], 2, 64, 16, seed=17)
    t = b.tables.clone()
    t[0, 1] = -7
    c = pkv.PagedTokens(b.pool, t, b.len_t)
    before = b.pool.clone()
    q, k, v = (randn((2, 2, 64), b.dtype, b.g) for _ in range(3))
    out = c.decode_append(k, v, q)
    with pytest.raises(pkv.KVError):
        c.check_device()
    kept, b.lens = b.lens, [16, 40]
    assert_attended(out, b, q)                      # token 16 has no page
    b.lens = [0, 40]
    assert_appended(b, before, [1, 1], k, v, None)
    b.lens = kept


# ---------------------------------------------------------------- as they are used together
@pytest.mark.parametrize("dtype,d,hkv,g,page", [("bf16", 128, 2, 4, 16), ("fp16", 64, 4, 1, 57)])
def test_prompts_then_tokens(pkv, dtype, d, hkv, g, page):
    """Prompts of unequal length appended at once, then steps, fused and apart, against dense attention over all keys."""
    dt, gn = DT[dtype], gen(18)
    prompts, steps = [37, 1, 90], 5
    rope = pkv.Rope(d, scaling="ntk", factor=2.0)
    width = -(-(max(prompts) + steps) // page)
    pool = torch.full((3 * width, 2, page, hkv, d), math.nan, dtype=dt, device="cuda")
    tables = torch.randperm(3 * width, generator=gn, device="cuda").to(torch.int32).view(3, width)
    lens = torch.tensor(prompts, dtype=torch.int32, device="cuda")
    cache = pkv.PagedTokens(pool, tables, lens)
    k, v = randn((sum(prompts), hkv, d), dt, gn), randn((sum(prompts), hkv, d), dt, gn)
    cache.append(k, v, cu_new=torch.tensor([0, 37, 38, 128], dtype=torch.int32, device="cuda"), rope=rope)
    b = Batch.__new__(Batch)
    b.pool, b.page, b.d, b.lens, b.rows = pool, page, d, list(prompts), tables.tolist()
    hold = [(k[a:e], v[a:e]) for a, e in ((0, 37), (37, 38), (38, 128))]
    for i in range(steps):
        lens += 1
        b.lens = [n + 1 for n in b.lens]
        q, k, v = randn((3, hkv * g, d), dt, gn), randn((3, hkv, d), dt, gn), randn((3, hkv, d), dt, gn)
        hold = [(torch.cat([a, k[s:s + 1]]), torch.cat([c, v[s:s + 1]])) for s, (a, c) in enumerate(hold)]
        if i % 2:
            out = cache.decode_append(k, v, q, rope=rope)
            exact_q = torch.tensor(turned(q, lens - 1, rope)[0], device="cuda")
        else:
            cache.append(k, v, rope=rope)
            exact_q = rope.rotate(q, lens - 1)
            out = cache.decode(exact_q)
        kv = []
        for s, (ks, vs) in enumerate(hold):
            p, r = b.where(s, torch.arange(b.lens[s], device="cuda"))
            assert_turned(pool[p, 0, r], ks, torch.arange(b.lens[s]), rope)
            kv.append((pool[p, 0, r].double(), vs.double()))
        assert_attended(out, b, exact_q, extra=2**-16 + ROT, kv=kv)
    cache.check_device()


def test_captured_steps_follow_the_lengths(pkv):
    """Two captured steps that share a workspace, replayed in turn while the lengths grow, against eager calls."""
    lens = [30, 0, 120, 16]
    b = Batch(pkv, [n + 40 if n else 0 for n in lens], 2, 128, 16, seed=19)
    eager = Batch(pkv, [n + 40 if n else 0 for n in lens], 2, 128, 16, seed=19)
    rope = pkv.Rope(128)
    for x in (b, eager):
        x.len_t.copy_(torch.tensor(lens, dtype=torch.int32))
    q, k, v = randn((4, 8, 128), b.dtype, b.g), randn((4, 2, 128), b.dtype, b.g), randn((4, 2, 128), b.dtype, b.g)
    ws = b.cache.workspace(8)
    side = torch.cuda.Stream()
    outs, graphs = [torch.zeros_like(q) for _ in range(2)], []
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        b.cache.decode_append(k, v, q, rope=rope, workspace=ws)     # warm
    torch.cuda.current_stream().wait_stream(side)
    eager.cache.decode_append(k, v, q, rope=rope)
    for i in range(2):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            if i:
                b.cache.append(k, v, rope=rope)
                b.cache.decode(rope.rotate(q, b.len_t - 1), out=outs[i], workspace=ws)
            else:
                b.cache.decode_append(k, v, q, rope=rope, out=outs[i], workspace=ws)
        graphs.append(graph)
    own = torch.zeros_like(q)                       # and one with a workspace of the graph's
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        own.copy_(b.cache.decode(q))
    for step in range(30):
        live = (b.len_t > 0).int()
        b.len_t += live
        eager.len_t += live
        k.copy_(randn(k.shape, b.dtype, b.g))
        q.copy_(randn(q.shape, b.dtype, b.g))
        graphs[step % 2].replay()
        if step % 2:
            eager.cache.append(k, v, rope=rope)
            want = eager.cache.decode(rope.rotate(q, eager.len_t - 1))
        else:
            want = eager.cache.decode_append(k, v, q, rope=rope)
        assert torch.equal(outs[step % 2], want), step
        graph.replay()
        assert torch.equal(own, eager.cache.decode(q)), step
    b.cache.check_device()


def test_unprepared_workspace_is_reported(pkv):
    b = Batch(pkv, [9000], 1, 64, 64, seed=23)
    q = randn((1, 2, 64), b.dtype, b.g)
    ws = torch.zeros(b.cache.workspace_bytes(2), dtype=torch.uint8, device="cuda")
    b.cache.decode(q, workspace=ws)
    with pytest.raises(pkv.KVError) as e:
        b.cache.check_device()
    assert e.value.name == "DEVICE_CHECK"
    pkv.kv_decode_workspace_init(b.cache._c, 2, ws.data_ptr(), ws.numel(), torch.cuda.current_stream().cuda_stream)
    assert_attended(b.cache.decode(q, workspace=ws), b, q)
    b.cache.check_device()


def test_one_workspace_for_all_heads(pkv):
    """A workspace of the largest call serves batches of other heads and lengths in turn."""
    batches = [Batch(pkv, [20000, 300], hkv, 64, 64, seed=29 + hkv) for hkv in (1, 3, 8)]
    calls = [(b, randn((2, b.hkv * g, 64), b.dtype, b.g)) for b in batches for g in (1, 5, 16)]
    most = max((b.cache.workspace_bytes(q.shape[1]), i) for i, (b, q) in enumerate(calls))[1]
    ws = calls[most][0].cache.workspace(calls[most][1].shape[1])
    for _ in range(2):
        for b, q in calls:
            assert torch.equal(b.cache.decode(q, workspace=ws), b.cache.decode(q))
    b, q = calls[0]
    assert_attended(b.cache.decode(q, workspace=ws), b, q)


@pytest.mark.parametrize("seqs,hkv,g,n", [(1, 1, 1, 70000), (1, 1, 16, 40000), (2, 1, 5, 30000), (5, 1, 3, 9000), (1, 3, 2, 20011)])
@pytest.mark.parametrize("d", [64, 128])
def test_many_parts(pkv, seqs, hkv, g, n, d):
    """Units of up to 296 parts: joined in one round and in two, full groups and ragged ones."""
    b = Batch(pkv, [n - 1000 * i for i in range(seqs)], hkv, d, 128, seed=24)
    q = randn((seqs, hkv * g, d), b.dtype, b.g)
    out = b.cache.decode(q, scale=0.3)              # weights peaked enough for every part's to matter
    assert_attended(out, b, q, scale=0.3)
    for _ in range(5):
        assert torch.equal(out, b.cache.decode(q, scale=0.3))
    b.cache.check_device()


def test_captured_gradient(pkv):
    rope, pos = pkv.Rope(64), torch.arange(50, device="cuda", dtype=torch.int32)
    x = torch.randn(50, 3, 64, device="cuda", requires_grad=True)
    dy = torch.randn(50, 3, 64, device="cuda")
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        torch.autograd.grad(rope.rotate(x, pos), x, dy)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y = rope.rotate(x, pos)
        dx, = torch.autograd.grad(y, x, dy)
    with torch.no_grad():
        x.copy_(torch.randn(50, 3, 64, device="cuda"))
    dy.copy_(torch.randn(50, 3, 64, device="cuda"))
    graph.replay()
    assert_turned(y, x, pos, rope)
    assert_turned(dx, dy, pos, rope, -1)


def test_streams(pkv):
    """An explicit stream, torch's or a raw one, and two calls at once with workspaces of their own."""
    b = Batch(pkv, [3000, 500], 2, 128, 64, seed=20)
    q = randn((2, 8, 128), b.dtype, b.g)
    want = b.cache.decode(q)
    torch.cuda.synchronize()
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    got = [b.cache.decode(q, stream=s) for _ in range(20) for s in (s1, s2, s1.cuda_stream)]
    torch.cuda.synchronize()
    assert all(torch.equal(x, want) for x in got)
    rope, pos = pkv.Rope(128), torch.arange(2, device="cuda", dtype=torch.int32)
    y = rope.rotate(q, pos, stream=s1)
    s1.synchronize()
    assert torch.equal(y, rope.rotate(q, pos))


def test_threads(pkv):
    """Calls of several host threads on one object, each on a stream of its own."""
    import threading
    b = Batch(pkv, [9000, 4000, 0, 70], 1, 64, 64, seed=28)
    rope, pos = pkv.Rope(64), torch.arange(4, device="cuda", dtype=torch.int32)
    qs = [randn((4, 3, 64), b.dtype, b.g) for _ in range(4)]
    want = [(b.cache.decode(q), rope.rotate(q, pos)) for q in qs]
    torch.cuda.synchronize()
    wrong = []

    def work(i):
        with torch.cuda.stream(torch.cuda.Stream()):
            for _ in range(50):
                got = b.cache.decode(qs[i]), rope.rotate(qs[i], pos)
                torch.cuda.current_stream().synchronize()
                if not all(torch.equal(x, y) for x, y in zip(got, want[i])):
                    wrong.append(i)

    threads = [threading.Thread(target=work, args=(i,)) for i in range(4)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not wrong
    b.cache.check_device()


def test_refused_calls(pkv):
    b = Batch(pkv, [10, 20], 2, 64, 16, seed=21)
    q, k = randn((2, 4, 64), b.dtype, b.g), randn((2, 2, 64), b.dtype, b.g)
    ws = torch.empty(100, dtype=torch.uint8, device="cuda")
    bad = [lambda: b.cache.decode(q[:1]), lambda: b.cache.decode(q[:, :3]), lambda: b.cache.decode(q.half()),
           lambda: b.cache.decode(q[0]), lambda: b.cache.decode(q[..., :32]), lambda: b.cache.decode(q.cpu()),
           lambda: b.cache.decode(q, out=q[:, :2]), lambda: b.cache.decode(q, out=torch.empty_like(q).half()),
           lambda: b.cache.decode(q, scale=0.0), lambda: b.cache.decode(q.float().requires_grad_().bfloat16()),
           lambda: b.cache.append(k[:1], k), lambda: b.cache.append(k, k.float()), lambda: b.cache.append(k[:, :1], k),
           lambda: b.cache.append(k, k, cu_new=torch.zeros(2, dtype=torch.int32, device="cuda")),
           lambda: b.cache.append(k, k, cu_new=torch.zeros(3, dtype=torch.int64, device="cuda")),
           lambda: b.cache.append(k, k, positions=torch.zeros(3, dtype=torch.int32, device="cuda")),
           lambda: b.cache.append(k.clone().requires_grad_(), k),
           lambda: b.cache.decode_append(k, k, q, positions=torch.zeros(2, dtype=torch.int32)),
           lambda: pkv.PagedTokens(b.pool, b.tables.long(), b.len_t), lambda: pkv.PagedTokens(b.pool[:, :, ::2], b.tables, b.len_t),
           lambda: pkv.PagedTokens(b.pool, b.tables, b.len_t[:1]), lambda: pkv.PagedTokens(b.pool, b.tables.cpu(), b.len_t),
           lambda: pkv.PagedTokens(b.pool, b.tables[0], b.len_t)]
    for call in bad:
        with pytest.raises(ValueError):
            call()
    for name in ("pool", "tables", "lens"):         # the library holds their addresses
        with pytest.raises(AttributeError):
            setattr(b.cache, name, getattr(b.cache, name).clone())
    with pytest.raises(pkv.KVError) as e:
        b.cache.decode(q, workspace=ws)
    assert e.value.name == "CAPACITY"
    with pytest.raises(pkv.KVError) as e:
        b.cache.decode(q, window=-1)
    assert e.value.name == "ARG"
    for call in (lambda: b.cache.decode(q), lambda: b.cache.decode_append(k, k, q), lambda: b.cache.append(k, k)):
        pkv.kv_testing_fail_launches(1)
        with pytest.raises(pkv.KVError) as e:
            call()
        assert e.value.name == "CUDA"
    assert_attended(b.cache.decode(q), b, q)


def test_a_scale_below_32_bits_is_refused(pkv):
    b = Batch(pkv, [10], 2, 64, 16, seed=22)
    for scale in (1e-60, -1e-60):
        with pytest.raises(ValueError):   # 0 would stand for the default
            b.cache.decode(randn((1, 2, 64), b.dtype, b.g), scale=scale)


def test_written_tensors_count_as_changed(pkv):
    """What autograd saved and a call then wrote: its backward pass says so, as for torch's own in-place calls."""
    b, rope = Batch(pkv, [10, 20], 2, 64, 16, seed=23), pkv.Rope(64)
    k, q, pos = randn((2, 2, 64), b.dtype, b.g), randn((2, 4, 64), b.dtype, b.g), b.len_t - 1
    x, out = randn((2, 2, 64), torch.float32, b.g), torch.empty_like(q)
    for saved, call in [(x, lambda: rope.rotate(x, pos, out=x)), (b.pool, lambda: b.cache.append(k, k)),
                        (b.pool, lambda: b.cache.decode_append(k, k, q)), (out, lambda: b.cache.decode(q, out=out))]:
        w = torch.ones((), device="cuda", dtype=saved.dtype, requires_grad=True)
        y = (saved * w).sum()
        call()
        with pytest.raises(RuntimeError, match="modified by an inplace operation"):
            y.backward()
    version = b.pool._version
    b.cache.decode(q)
    assert b.pool._version == version
    with torch.inference_mode():   # its tensors have no versions
        z = x * 1
        rope.rotate(z, pos, out=z)
        b.cache.decode(q * 1, out=q * 1)


def test_tensors_that_stand_for_others_are_refused(pkv):
    b, rope = Batch(pkv, [10, 20], 2, 64, 16, seed=24), pkv.Rope(64)
    k, q, pos = randn((2, 2, 64), b.dtype, b.g), randn((2, 4, 64), b.dtype, b.g), b.len_t - 1
    wide = torch.empty((2, 1, 64), device="cuda").expand(2, 3, 64)
    for call in (lambda: rope.rotate(wide, pos, out=wide), lambda: rope.rotate(torch.empty(2, 3, 64, device="cuda"), pos, out=wide),
                 lambda: rope.rotate(torch._neg_view(wide.contiguous()), pos), lambda: b.cache.decode(torch._neg_view(q)),
                 lambda: b.cache.append(k, torch._neg_view(k)), lambda: b.cache.decode(q, out=torch.empty_like(q).requires_grad_())):
        with pytest.raises(ValueError):
            call()
    b.pool.requires_grad_()
    for call in (lambda: b.cache.decode(q), lambda: b.cache.append(k, k), lambda: b.cache.decode_append(k, k, q)):
        with pytest.raises(ValueError):
            call()
    with torch.no_grad():
        assert_attended(b.cache.decode(q), b, q)


# ---------------------------------------------------------------- over a frame plan's pages
@pytest.mark.parametrize("ps,d,dtype,frames", [(16, 64, "bf16", 12), (130, 128, "fp16", 7)])
def test_decode_over_a_frame_plan(pkv, ps, d, dtype, frames):
    """One token of the frame at a time against what kv_run's frame sees: the frame path's tolerance, and the 64-bit form's."""
    from gpu_drive import MAX_ABS, MEAN_ABS
    s, h, ns = 2, 3, 6
    caches = pkv.PagedKVCache.group(s, 60, ps, h, d, scale_frames=2, window=3, num_special=ns, dtype=dtype)
    caches[0].allocate_pools("cuda")
    g = gen(22)
    qs = []
    for f in range(frames):
        qs = []
        for i, c in enumerate(caches):
            if f < frames - 2 or i == 0:
                x = randn((3, ps + ns, h, d), DT[dtype], g)
                c.append_frame(0, x[1], x[2])
                c.evict_frames()
            qs.append(randn((ps + ns, h, d), DT[dtype], g))
    ws = torch.empty(pkv.workspace_bytes(caches), dtype=torch.uint8, device="cuda")
    plan = pkv.Plan(caches, ws)
    want = plan.run(0, torch.cat(qs)).view(s, ps + ns, h, d)
    cache = pkv.PagedTokens.of_plan(plan, 0)
    for t in (0, ps + ns - 1):
        q = torch.stack([x[t] for x in qs])
        out = cache.decode(q)
        diff = (out.float() - want[:, t].float()).abs()
        assert diff.max() <= MAX_ABS and diff.mean() <= MEAN_ABS
        b = Batch.__new__(Batch)
        b.pool, b.page, b.d = cache.pool, ps, d
        b.rows, b.lens = cache.tables.tolist(), cache.lens.tolist()
        assert_attended(out, b, q)
    cache.check_device()
    one = pkv.PagedTokens.of_plan(plan, 0, streams=[1])
    assert torch.equal(one.decode(qs[1][:1]), cache.decode(torch.stack([qs[0][0], qs[1][0]]))[1:])


def test_plans_with_hidden_tokens_are_refused(pkv):
    c = pkv.PagedKVCache(30, 16, 2, 64, scale_frames=1, window=2, camera_only=True)
    c.allocate_pools("cuda")
    x = torch.zeros(22, 2, 64, dtype=torch.bfloat16, device="cuda")
    c.append_frame(0, x, x)
    plan = pkv.Plan([c])
    with pytest.raises(ValueError):
        pkv.PagedTokens.of_plan(plan, 0)
    other = pkv.PagedKVCache(30, 16, 2, 64, scale_frames=1, window=2)
    other.allocate_pools("cuda")
    other.append_frame(0, x, x)
    d = pkv.PagedKVCache(30, 16, 2, 64, scale_frames=1, window=2)
    d.allocate_pools("cuda")
    d.append_frame(0, x, x)
    with pytest.raises(ValueError):
        pkv.PagedTokens.of_plan(pkv.Plan([other, d]), 0)
    assert pkv.PagedTokens.of_plan(pkv.Plan([other, d]), 0, streams=[1]).lens.tolist() == [22]
