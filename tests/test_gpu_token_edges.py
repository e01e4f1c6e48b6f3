"""Token operators on the GPU at the borders of what their documentation allows."""
import math

import numpy as np
import pytest
import torch

from test_gpu_tokens import DT, ROT, Batch, assert_appended, assert_attended, attended, gen, half_step, pkv, randn, turned  # noqa: F401

pytestmark = pytest.mark.gpu


def bits(x):
    return x.view(torch.int16)


# ---------------------------------------------------------------- lengths past the table
@pytest.mark.parametrize("held,hkv,g,d,page,dtype,window", [
    (64, 2, 1, 64, 16, "bf16", 0), (64, 1, 9, 128, 16, "fp16", 0), (20000, 2, 2, 64, 32, "bf16", 0),
    (9000, 1, 4, 128, 1000, "fp16", 777)])
def test_a_step_past_the_table_writes_nothing(pkv, held, hkv, g, d, page, dtype, window):
    """A length that the table cannot hold: its new token has no slot. It is not written, and what is attended to are the
    tokens that the table names, as they are in the pool."""
    b = Batch(pkv, [held, 40, held], hkv, d, page, dtype, seed=31)
    q = randn((3, hkv * g, d), b.dtype, b.g)
    k, v = randn((3, hkv, d), b.dtype, b.g), randn((3, hkv, d), b.dtype, b.g)
    for long in (held + 1, 2**31 - 1):
        before = b.pool.clone()
        b.len_t.copy_(torch.tensor([long, 40, -1], dtype=torch.int32))
        out = b.cache.decode_append(k, v, q, window=window)
        with pytest.raises(pkv.KVError) as e:
            b.cache.check_device()
        assert e.value.name == "DEVICE_CHECK"
        b.lens = [0, 40, 0]                         # only the second one's token is written
        assert_appended(b, before, [1, 1, 1], k, v, None)
        b.lens = [held, 40, 0]
        assert_attended(out, b, q, window=window)


# ---------------------------------------------------------------- weights far below the largest
@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
@pytest.mark.parametrize("d,g,fused", [(64, 1, False), (128, 4, False), (64, 16, False), (128, 2, True)])
def test_weights_far_below_the_largest(pkv, dtype, d, g, fused):
    """A key that takes nearly all of the weight and whose value is zero: the output is what the others' weights leave.
    Both the weights' sum and their products have to hold them: 2^-38 of the largest weight is the least that fp16 pools
    resolve (decode.cuh), a term per token."""
    gaps = [6, 8, 10, 11, 12, 13, 14, 15, 16]       # in units of e: the others' weights are e^-gap each
    b = Batch(pkv, [2048 + 37 * i for i in range(len(gaps))], 8, d, 64, dtype, seed=32)
    b.pool.zero_()
    for s, gap in enumerate(gaps):
        n = b.lens[s]
        j = torch.arange(n, device="cuda")
        p, r = b.where(s, j)
        v = (64 + 32 * torch.rand((n, 8, d), generator=b.g, device="cuda")).to(b.dtype)
        k = (randn((n, 8, d), b.dtype, b.g) * 2**-6).to(b.dtype)
        sink = j % 512 == 3                         # in every warp's share
        k[sink] = 0
        k[sink, :, 0] = gap * math.sqrt(d) / 8
        v[sink] = 0
        b.pool[p, 0, r], b.pool[p, 1, r] = k, v
    q = torch.zeros((len(gaps), 8 * g, d), dtype=b.dtype, device="cuda")
    q[..., 0] = 8
    q[..., 1:] = randn((len(gaps), 8 * g, d - 1), b.dtype, b.g) * 2**-4
    if fused:
        last = [b.where(s, torch.tensor([n - 1], device="cuda")) for s, n in enumerate(b.lens)]
        new = [torch.cat([b.pool[p, x, r] for p, r in last]) for x in (0, 1)]
        out = b.cache.decode_append(new[0], new[1], q)
    else:
        out = b.cache.decode(q)
    b.cache.check_device()
    eps, tiny = half_step(b.dtype)
    for s, n in enumerate(b.lens):
        k, v = b.kv(s, n)
        want, w, flat, most, seen = attended(k, v, q[s].double(), d ** -0.5, 0)
        assert float(want.abs().min()) > 0
        rel = most * d * 2**-23 + 2**-16 + (seen / 16 + 64) * 2**-23
        tol = eps * want.abs() + tiny + 2 * rel * w * (1 + eps) + flat * 2**-38
        err = (out[s].double() - want).abs()
        assert bool((err <= tol).all()), f"gap {gaps[s]}: worst {float((err / tol).max()):.1f} of what is allowed"


# ---------------------------------------------------------------- infinities in masked places
@pytest.mark.parametrize("bad", [math.inf, -math.inf, math.nan])
@pytest.mark.parametrize("d,g", [(64, 2), (128, 16)])
def test_a_new_token_without_a_page_counts_for_nothing(pkv, bad, d, g):
    """Its key and value, infinite ones too, reach no output."""
    b = Batch(pkv, [17, 40, 5000], 2, d, 16, seed=33)
    t = b.tables.clone()
    t[0, 1] = -7
    t[2, 4999 // 16] = b.pool.shape[0]
    c = pkv.PagedTokens(b.pool, t, b.len_t)
    q = randn((3, 2 * g, d), b.dtype, b.g)
    k, v = randn((3, 2, d), b.dtype, b.g), randn((3, 2, d), b.dtype, b.g)
    k[0], v[0], k[2], v[2] = bad, bad, bad, bad
    out = c.decode_append(k, v, q)
    with pytest.raises(pkv.KVError):
        c.check_device()
    b.lens = [16, 40, 4992]
    assert_attended(out, b, q, extra=2**-16)


@pytest.mark.parametrize("lens,hkv,g,d,dtype", [
    ([1], 1, 1, 64, "bf16"), ([300, 7], 2, 3, 128, "fp16"), ([20000], 1, 16, 64, "fp16"), ([30000] * 3, 1, 1, 64, "bf16")])
def test_scores_that_are_all_minus_infinity(pkv, lens, hkv, g, d, dtype):
    """A softmax over nothing but -inf has no value; with a finite score among them the others have no weight. (Zeros are
    for rows that see no token.)"""
    b = Batch(pkv, lens, hkv, d, 64, dtype, seed=34)
    q = randn((len(lens), hkv * g, d), b.dtype, b.g).abs() + 0.1
    keep = b.pool.clone()
    for s, n in enumerate(lens):
        p, r = b.where(s, torch.arange(n, device="cuda"))
        b.pool[p, 0, r] = -math.inf
    assert bool(b.cache.decode(q).isnan().all())
    some = [max(1, n // 3) for n in lens]            # the first third as it was
    kv = []
    for s, n in enumerate(some):
        p, r = b.where(s, torch.arange(n, device="cuda"))
        b.pool[p, 0, r] = keep[p, 0, r]
        kv.append(b.kv(s, n))
    out = b.cache.decode(q)
    c = Batch.__new__(Batch)
    c.lens, c.d = some, d
    assert_attended(out, c, q, kv=kv)
    b.len_t.zero_()
    assert bool((b.cache.decode(q) == 0).all())
    b.cache.check_device()


@pytest.mark.parametrize("amplitude", [None, 3.0, 1e4])
@pytest.mark.parametrize("layout,d,g", [("half", 64, 1), ("interleaved", 128, 16)])
def test_rotated_queries_past_the_types_range(pkv, amplitude, layout, d, g):
    """In the step a rotated query is not rounded to the pool's type: values that fp16 does not reach count as they are."""
    b = Batch(pkv, [200, 3000], 2, d, 64, "fp16", seed=35)
    for s, n in enumerate(b.lens):
        p, r = b.where(s, torch.arange(n, device="cuda"))
        b.pool[p, 0, r] *= 2**-8
    rope = pkv.Rope(d, layout=layout, inv_freq=[0.7 + 0.01 * i for i in range(d // 2)], amplitude=amplitude)
    q = (randn((2, 2 * g, d), b.dtype, b.g).sign() * 60000).to(b.dtype)
    k, v = randn((2, 2, d), b.dtype, b.g) * 2**-14, randn((2, 2, d), b.dtype, b.g)
    pos = torch.tensor([3, 70001], dtype=torch.int32, device="cuda")
    scale = 2**-9 / (amplitude or 1)
    out = b.cache.decode_append(k, v, q, rope=rope, positions=pos, scale=scale)
    b.cache.check_device()
    exact_q = torch.tensor(turned(q, pos, rope)[0], device="cuda")
    assert float(exact_q.abs().max()) > 65504
    assert_attended(out, b, exact_q, scale=scale, extra=2**-16 + ROT)


# ---------------------------------------------------------------- derivatives and overlaps
def test_a_negated_gradient(pkv):
    rope, pos = pkv.Rope(64), torch.arange(5, device="cuda", dtype=torch.int32)
    x = torch.randn(5, 2, 64, device="cuda", requires_grad=True)
    dy = torch.randn(5, 2, 64, device="cuda")
    want, = torch.autograd.grad(rope.rotate(x, pos), x, -dy)
    got, = torch.autograd.grad(rope.rotate(x, pos), x, torch._neg_view(dy))
    assert torch.equal(got, want)


def test_forward_mode_is_refused(pkv):
    """No operator has a forward-mode derivative: a tangent is refused, not dropped."""
    import torch.autograd.forward_ad as fwd
    b, rope = Batch(pkv, [10, 20], 2, 64, 16, seed=36), pkv.Rope(64)
    k, q, pos = randn((2, 2, 64), b.dtype, b.g), randn((2, 4, 64), b.dtype, b.g), b.len_t - 1
    x = randn((2, 3, 64), torch.float32, b.g)
    with fwd.dual_level():
        dual = lambda y: fwd.make_dual(y, torch.ones_like(y))  # noqa: E731
        for call in (lambda: rope.rotate(dual(x), pos), lambda: rope.rotate(x, pos, out=dual(x.clone())),
                     lambda: b.cache.decode(dual(q)), lambda: b.cache.append(k, dual(k)),
                     lambda: b.cache.decode_append(dual(k), k, q), lambda: b.cache.decode(q, out=dual(torch.empty_like(q)))):
            with pytest.raises(ValueError, match="tangent"):
                call()
        with pytest.raises((RuntimeError, ValueError)):
            rope.rotate(dual(x.clone().requires_grad_()), pos)
        rope.rotate(x, pos)
        b.cache.decode(q)


def test_outputs_that_overlap_inputs_are_refused(pkv):
    """`out` is x (or q) itself or apart from every input; what lies in the same memory and is neither is refused."""
    b, rope = Batch(pkv, [10, 20], 2, 64, 16, seed=37, poison=False), pkv.Rope(64)
    pos = b.len_t - 1
    buf = randn((40, 64), torch.float32, b.g)
    x, wide, flat = buf[:6].view(2, 3, 64), buf.view(2, 20, 64), buf.view(-1)
    for a, out in ((x, buf[1:7].view(2, 3, 64)), (x, buf[5:11].view(2, 3, 64)), (x, flat[2:386].view(2, 3, 64)),
                   (x, flat[383:767].view(2, 3, 64)), (wide[:, 2:5], wide[:, 4:7]), (wide[:, 2:5], wide[:, :3]),
                   (wide[:, :3], x), (x, wide[:, :3]), (wide[:, :3], buf[21:27].view(2, 3, 64))):
        with pytest.raises(ValueError, match="memory"):
            rope.rotate(a, pos, out=out)
    want = rope.rotate(wide[:, 2:5], pos)
    rope.rotate(wide[:, 2:5], pos, out=wide[:, 5:8])    # other heads of the same rows
    assert torch.equal(wide[:, 5:8], want)
    rope.rotate(wide[:, 2:5], pos, out=buf[8:14].view(2, 3, 64))   # between the rows
    assert torch.equal(buf[8:14].view(2, 3, 64), want)
    assert torch.equal(rope.rotate(wide[:, 2:5], pos, out=wide[:, 2:5]), want)
    q, k = randn((2, 4, 64), b.dtype, b.g), randn((2, 2, 64), b.dtype, b.g)
    row, pad = b.pool.view(-1, 64), randn((30, 64), b.dtype, b.g)
    inside = row[8:12].view(2, 2, 64)
    for call in (lambda: b.cache.append(inside, k), lambda: b.cache.append(k, inside), lambda: b.cache.decode_append(inside, k, q),
                 lambda: b.cache.decode_append(k, inside, q), lambda: b.cache.decode_append(k, k, row[:8].view(2, 4, 64)),
                 lambda: b.cache.decode(q, out=row[:8].view(2, 4, 64)), lambda: b.cache.decode_append(k, k, q, out=row[:8].view(2, 4, 64)),
                 lambda: b.cache.decode(pad[:8].view(2, 4, 64), out=pad[4:12].view(2, 4, 64)),
                 lambda: b.cache.decode_append(pad[:4].view(2, 2, 64), k, q, out=pad[2:10].view(2, 4, 64)),
                 lambda: b.cache.decode_append(k, pad[9:13].view(2, 2, 64), q, out=pad[2:10].view(2, 4, 64))):
        with pytest.raises(ValueError, match="memory"):
            call()
    heads = pad.view(2, 15, 64)[:, :4]
    want = b.cache.decode(heads)
    assert torch.equal(b.cache.decode(heads, out=pad[5:13].view(2, 4, 64)), want)
    assert torch.equal(b.cache.decode(row[8:16].view(2, 4, 64)), b.cache.decode(row[8:16].view(2, 4, 64).clone()))
    want = b.cache.decode(q)
    assert torch.equal(b.cache.decode(q, out=q), want)


# ---------------------------------------------------------------- appending
def test_a_cu_new_past_the_tokens_given_is_reported(pkv):
    """Tokens that cu_new counts and the call does not bring: those that it brings are written, the lack is reported."""
    b = Batch(pkv, [20, 20, 20], 2, 64, 8, seed=38)
    k, v = randn((7, 2, 64), b.dtype, b.g), randn((7, 2, 64), b.dtype, b.g)
    for cu, ok in (([0, 3, 3, 7], True), ([0, 3, 3, 8], False), ([0, 3, 9, 9], False), ([0, 3, 7, 2000000000], False),
                   ([0, 2, 3, 5], True)):
        b.cache.append(k, v, cu_new=torch.tensor(cu, dtype=torch.int32, device="cuda"))
        if ok:
            b.cache.check_device()
        else:
            with pytest.raises(pkv.KVError) as e:
                b.cache.check_device()
            assert e.value.name == "DEVICE_CHECK"
    many = Batch(pkv, [1] * 1500, 1, 64, 4, seed=39)   # more sequences than are searched in shared memory
    cu = torch.arange(1501, dtype=torch.int32, device="cuda")
    x = randn((1500, 1, 64), many.dtype, many.g)
    many.cache.append(x, x, cu_new=cu)
    many.cache.check_device()
    with pytest.raises(pkv.KVError):
        many.cache.append(x[:1499], x[:1499], cu_new=cu)
        many.cache.check_device()


# ---------------------------------------------------------------- frame plans
def frames(pkv, n, ps=16, streams=1, **kw):
    caches = pkv.PagedKVCache.group(streams, 40 * streams, ps, 2, 64, scale_frames=1, window=3, num_special=4, **kw)
    caches[0].allocate_pools("cuda")
    g = gen(40)
    for _ in range(n):
        for c in caches:
            for block in range(c.num_blocks):
                x = randn((2, ps + 4, 2, 64), DT[c.dtype], g)
                c.append_frame(block, x[0], x[1])
            c.evict_frames()
    return caches


def test_tokens_of_a_plan_are_read_only(pkv):
    """The pages are the caches': a token has no slot of its own there."""
    caches = frames(pkv, 6, streams=2)
    seqs = pkv.PagedTokens.of_plan(pkv.Plan(caches), 0)
    before = caches[0].pools[0].clone()
    q = torch.ones((2, 2, 64), dtype=torch.bfloat16, device="cuda")
    want = seqs.decode(q)
    for _ in range(2):
        for call in (lambda: seqs.append(q, q), lambda: seqs.decode_append(q, q, q),
                     lambda: seqs.append(q, q, cu_new=torch.tensor([0, 1, 2], dtype=torch.int32, device="cuda"))):
            with pytest.raises(ValueError, match="read"):
                call()
        seqs.lens.add_(1)
    assert torch.equal(bits(caches[0].pools[0]), bits(before))
    seqs.lens.sub_(2)
    assert torch.equal(seqs.decode(q), want)
    seqs.check_device()


def test_a_plans_pool_is_read_in_the_caches_type(pkv):
    """bind_pool takes any tensor of enough bytes: the cache's dtype is what its values are."""
    caches = frames(pkv, 4, dtype="fp16")
    q = randn((1, 2, 64), torch.float16, gen(41))
    want = pkv.PagedTokens.of_plan(pkv.Plan(caches), 0).decode(q)
    pool = caches[0].pools[0]
    for other in (pool.view(torch.bfloat16), pool.view(torch.uint8), pool.view(-1).view(torch.float32)):
        caches[0].pools[0] = other
        assert torch.equal(pkv.PagedTokens.of_plan(pkv.Plan(caches), 0).decode(q), want)


# ---------------------------------------------------------------- parts of four-warp launches
@pytest.mark.parametrize("n", [60000, 250000])
@pytest.mark.parametrize("d,g,fused", [(64, 1, False), (128, 8, False), (64, 11, False), (128, 16, False), (64, 2, True), (128, 9, True)])
def test_one_long_sequence_among_short_ones(pkv, n, d, g, fused):
    """As many sequences as launches of four-warp CTAs take, one of them in more parts than are joined at once: the
    sequences cut into parts where these suffice, else cut anywhere along the line."""
    lens = [1 + i % 5 for i in range(80)]
    lens[17] = n
    lens[3] = 0
    b = Batch(pkv, lens, 1, d, 500, seed=42 + g, dtype="bf16" if d == 64 else "fp16")
    q = randn((80, g, d), b.dtype, b.g)
    call = lambda: b.cache.decode(q, scale=0.3)  # noqa: E731
    if fused:
        k, v = randn((80, 1, d), b.dtype, b.g), randn((80, 1, d), b.dtype, b.g)
        call = lambda: b.cache.decode_append(k, v, q, scale=0.3)  # noqa: E731
    out = call()
    assert_attended(out, b, q, scale=0.3, extra=2**-16 if fused else 0.0)
    for _ in range(5):
        assert torch.equal(out, call())
    b.cache.check_device()
