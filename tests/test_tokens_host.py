"""Token operators on the host: refusals, frequencies, and models of the index
arithmetic that the kernels use. No GPU, no launches."""
import ctypes
import math
import os
import random
import shutil
import subprocess

import pytest

HERE = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(HERE, "..", "paged_kv_cache_frame_b200", "csrc")


@pytest.fixture(scope="module")
def pkv():
    from paged_kv_cache_frame_b200 import build
    build.build()
    import paged_kv_cache_frame_b200 as m
    return m


def code(pkv, f, *args):
    with pytest.raises(pkv.KVError) as e:
        f(*args)
    return e.value.name


# ---------------------------------------------------------------- frequencies
def theta(rot, base, scaling, factor=1.0, context=0.0, low=1.0, high=32.0):
    out = []
    for i in range(rot // 2):
        t = base ** (-2 * i / rot)
        if scaling == "linear":
            t = t / factor
        if scaling == "ntk":
            # another base, such that the last pair turns `factor` times slower
            t = (base * factor ** (rot / (rot - 2))) ** (-2 * i / rot) if rot > 2 else t
        if scaling == "yarn":
            turns = context * t / (2 * math.pi)
            g = min(1.0, max(0.0, (turns - low) / (high - low)))
            t = (1 - g) * t / factor + g * t
        out.append(t)
    return out


@pytest.mark.parametrize("rot,scaling,kw", [
    (128, "none", {}), (2, "none", {}), (2, "ntk", {"factor": 8.0}), (64, "linear", {"factor": 2.5}),
    (256, "ntk", {"factor": 16.0}), (96, "yarn", {"factor": 4.0, "context": 4096}),
    (48, "yarn", {"factor": 8.0, "context": 1024, "low": 1.0, "high": 4.0})])
def test_frequencies(pkv, rot, scaling, kw):
    r = pkv.Rope(rot, base=5e5, scaling=scaling, factor=kw.get("factor", 1.0), original_context=kw.get("context", 0),
                 low_turns=kw.get("low", 1.0), high_turns=kw.get("high", 32.0))
    assert r.inv_freq == pytest.approx(theta(rot, 5e5, scaling, **kw), rel=1e-14)
    assert r.amplitude == pytest.approx(0.1 * math.log(kw["factor"]) + 1 if scaling == "yarn" else 1.0, rel=1e-15)


def test_given_frequencies_and_amplitude(pkv):
    r = pkv.Rope(6, layout="interleaved", inv_freq=[1.0, -0.25, 7.5], amplitude=1.25)
    assert (r.inv_freq, r.amplitude, r.rot_dim, r.layout) == ([1.0, -0.25, 7.5], 1.25, 6, "interleaved")
    assert pkv.Rope(8, scaling="yarn", factor=4.0, original_context=64, amplitude=1.0).amplitude == 1.0


@pytest.mark.parametrize("kw", [
    {"rot_dim": 0}, {"rot_dim": 3}, {"rot_dim": 258}, {"rot_dim": 64, "base": 0.0}, {"rot_dim": 64, "base": math.nan},
    {"rot_dim": 64, "scaling": "linear", "factor": 0.0}, {"rot_dim": 64, "scaling": "yarn", "factor": 2.0},
    {"rot_dim": 64, "scaling": "yarn", "factor": 2.0, "original_context": 64, "low_turns": 4.0, "high_turns": 4.0},
    {"rot_dim": 4, "inv_freq": [1.0, math.inf]}, {"rot_dim": 4, "inv_freq": [1.0, 2e6]},
    {"rot_dim": 4, "inv_freq": [1.0, 0.5], "amplitude": math.inf}])
def test_rope_refusals(pkv, kw):
    assert code(pkv, lambda: pkv.Rope(**kw)) == "ARG"


@pytest.mark.parametrize("amplitude", [1e300, 3.5e38, 1e-60, 1e-46])
def test_amplitudes_that_do_not_fit_32_bits_are_refused(pkv, amplitude):
    """The kernels' factor would be infinite, or 0."""
    assert code(pkv, lambda: pkv.Rope(8, amplitude=amplitude)) == "ARG"
    assert code(pkv, lambda: pkv.Rope(4, inv_freq=[1.0, 0.5], amplitude=amplitude)) == "ARG"


@pytest.mark.parametrize("kw", [
    {"rot_dim": 4, "layout": "thirds"}, {"rot_dim": 4, "scaling": "cubic"}, {"rot_dim": 4, "amplitude": 0.0},
    {"rot_dim": 4, "amplitude": math.nan}, {"rot_dim": 4, "inv_freq": [1.0]},
    {"rot_dim": 2, "inv_freq": [1.0], "scaling": "ntk", "factor": 2.0}])
def test_rope_argument_errors(pkv, kw):
    with pytest.raises(ValueError):
        pkv.Rope(**kw)


def test_rope_c_refusals(pkv):
    L = pkv.capi.lib()
    d = (ctypes.c_double * 1)(1.0)
    assert L.kv_rope_init_frequencies(None, 2, 0, d, 1.0) == pkv.capi.KV_ERR_ARG
    h = ctypes.c_void_p()
    assert L.kv_rope_init_frequencies(ctypes.byref(h), 2, 0, None, 1.0) == pkv.capi.KV_ERR_ARG
    assert L.kv_rope_init_frequencies(ctypes.byref(h), 2, 5, d, 1.0) == pkv.capi.KV_ERR_ARG
    assert h.value is None
    L.kv_rope_free(None)
    assert L.kv_rope_get(None, None, None, None, None, 0) == pkv.capi.KV_ERR_ARG


# ---------------------------------------------------------------- refusals before any launch
def rows(pkv, at=4096, token=128, head=64):
    return pkv.capi.kv_rows(at, token, head)


def tokens(pkv, **kw):
    """A batch whose addresses are never followed: every call here is refused
    or has nothing to do."""
    f = dict(pool=4096, tables=4096, lens=4096, error=4096, table_stride=4, max_pages=8, page_size=16, num_heads=2,
             head_dim=64, dtype=pkv.KV_BF16, table_width=4, n_seqs=3)
    f.update(kw)
    return pkv.capi.kv_tokens(**f)


BAD_TOKENS = [
    ({"head_dim": 96}, "UNSUPPORTED"), ({"dtype": 2}, "UNSUPPORTED"), ({"dtype": -1}, "UNSUPPORTED"),
    ({"max_pages": 0}, "ARG"), ({"page_size": 0}, "ARG"), ({"num_heads": 0}, "ARG"), ({"num_heads": 9000}, "ARG"),
    ({"n_seqs": -1}, "ARG"), ({"n_seqs": 16385}, "ARG"), ({"table_width": 0}, "ARG"), ({"table_stride": 3}, "ARG"),
    ({"pool": None}, "ARG"), ({"pool": 4104}, "ARG"), ({"tables": None}, "ARG"), ({"lens": None}, "ARG"),
    ({"error": None}, "ARG"), ({"error": 4098}, "ARG"), ({"tables": 4097}, "ARG"),
    ({"table_width": 1 << 20, "table_stride": 1 << 20, "page_size": 1025}, "ARG"),
    ({"max_pages": 1 << 20, "page_size": 1024}, "ARG")]


@pytest.mark.parametrize("kw,want", BAD_TOKENS, ids=lambda x: str(x))
def test_sequence_refusals(pkv, kw, want):
    c, r = tokens(pkv, **kw), rows(pkv)
    assert code(pkv, pkv.kv_append_tokens, c, r, r, 3) == want
    assert code(pkv, pkv.kv_decode, c, r, 2, 0.0, 0, 4096, 4096, 1 << 30) == want
    assert code(pkv, pkv.kv_decode_append, c, r, r, r, 2, None, None, 0.0, 0, 4096, 4096, 1 << 30) == want
    assert pkv.kv_decode_workspace_bytes(c, 2) == 0


def test_append_refusals(pkv):
    c, r = tokens(pkv), rows(pkv)
    wide = pkv.Rope(128)
    for args in [(None, r, r, 3), (c, r, r, -1), (c, r, r, 4), (c, None, r, 3), (c, r, None, 3),
                 (c, rows(pkv, at=None), r, 3), (c, rows(pkv, at=4100), r, 3), (c, r, rows(pkv, token=132), 3),
                 (c, r, rows(pkv, head=68), 3), (c, r, r, 3, 4098), (c, r, r, 3, None, None, 4098),
                 (c, r, r, 3, None, wide.handle)]:
        assert code(pkv, pkv.kv_append_tokens, *args) == "ARG"


def test_decode_refusals(pkv):
    c, r = tokens(pkv), rows(pkv)
    wide, big = pkv.Rope(128), 1 << 30
    need = pkv.kv_decode_workspace_bytes(c, 2)
    assert need > 0
    assert code(pkv, pkv.kv_decode, c, r, 2, 0.0, 0, 4096, 4096, need - 1) == "CAPACITY"
    for args in [(None, r, 2, 0.0, 0, 4096, 4096, big), (c, None, 2, 0.0, 0, 4096, 4096, big),
                 (c, r, 0, 0.0, 0, 4096, 4096, big), (c, r, 3, 0.0, 0, 4096, 4096, big),
                 (c, r, 8194, 0.0, 0, 4096, 4096, big), (c, r, 2, math.inf, 0, 4096, 4096, big),
                 (c, r, 2, math.nan, 0, 4096, 4096, big), (c, r, 2, 0.0, -1, 4096, 4096, big),
                 (c, r, 2, 0.0, 0, None, 4096, big), (c, r, 2, 0.0, 0, 4098, 4096, big),
                 (c, r, 2, 0.0, 0, 4096, None, big), (c, r, 2, 0.0, 0, 4096, 4104, big),
                 (c, rows(pkv, at=4098), 2, 0.0, 0, 4096, 4096, big), (c, rows(pkv, head=66), 2, 0.0, 0, 4096, 4096, big)]:
        assert code(pkv, pkv.kv_decode, *args) == "ARG"
    for k, v, rope, pos in [(None, r, None, None), (r, None, None, None), (r, r, wide.handle, None),
                            (r, r, None, 4098), (rows(pkv, at=4104), r, None, None)]:
        assert code(pkv, pkv.kv_decode_append, c, k, v, r, 2, rope, pos, 0.0, 0, 4096, 4096, big) == "ARG"
    assert code(pkv, pkv.kv_tokens_check, None) == "ARG"
    assert pkv.kv_decode_workspace_bytes(c, 3) == 0
    for args, want in [((None, 2, 4096, big), "ARG"), ((c, 3, 4096, big), "ARG"), ((c, 2, None, big), "ARG"),
                       ((c, 2, 4104, big), "ARG"), ((c, 2, 4096, need - 1), "CAPACITY")]:
        assert code(pkv, pkv.kv_decode_workspace_init, *args) == want


def test_rotate_refusals(pkv):
    r, x = pkv.Rope(64), rows(pkv)
    for args, want in [((None, x, x, 4096, 3, 2, 64, 0), "ARG"), ((r.handle, None, x, 4096, 3, 2, 64, 0), "ARG"),
                       ((r.handle, x, None, 4096, 3, 2, 64, 0), "ARG"), ((r.handle, x, x, None, 3, 2, 64, 0), "ARG"),
                       ((r.handle, x, x, 4098, 3, 2, 64, 0), "ARG"), ((r.handle, x, x, 4096, -1, 2, 64, 0), "ARG"),
                       ((r.handle, x, x, 4096, 3, -1, 64, 0), "ARG"), ((r.handle, x, x, 4096, 3, 2, 62, 0), "ARG"),
                       ((r.handle, x, x, 4096, 3, 2, 65, 0), "ARG"), ((r.handle, x, x, 4096, 3, 2, 514, 0), "ARG"),
                       ((r.handle, rows(pkv, at=4097), x, 4096, 3, 2, 64, 0), "ARG"),
                       ((r.handle, x, rows(pkv, at=4098), 4096, 3, 2, 64, 2), "ARG"),
                       ((r.handle, x, rows(pkv, token=256), 4096, 3, 2, 64, 0), "ARG"),
                       ((r.handle, x, x, 4096, 3, 2, 64, 3), "UNSUPPORTED")]:
        assert code(pkv, pkv.kv_rotate, *args) == want


def test_nothing_to_do_launches_nothing(pkv):
    r, x = pkv.Rope(64), rows(pkv)
    nul = rows(pkv, at=None)
    pkv.kv_testing_fail_launches(1)   # a launch would take this one and fail
    try:
        pkv.kv_rotate(r.handle, nul, nul, None, 0, 2, 64, 0)
        pkv.kv_rotate(r.handle, nul, nul, None, 3, 0, 64, 0)
        pkv.kv_append_tokens(tokens(pkv), nul, nul, 0, 4096)
        c = tokens(pkv, n_seqs=0, tables=None, lens=None)
        pkv.kv_append_tokens(c, nul, nul, 0)
        pkv.kv_decode(c, nul, 2, 0.0, 0, None, None, 0)
        pkv.kv_decode_append(c, nul, nul, nul, 2, r.handle, None, 0.0, 0, None, None, 0)
        assert code(pkv, pkv.kv_append_tokens, tokens(pkv), x, x, 3) == "CUDA"
    finally:
        pkv.kv_testing_fail_launches(0)


def test_failing_launches_are_reported(pkv):
    c, r, x = tokens(pkv), pkv.Rope(64), rows(pkv)
    big = 1 << 30
    for call in [lambda: pkv.kv_rotate(r.handle, x, x, 4096, 3, 2, 64, 0),
                 lambda: pkv.kv_append_tokens(c, x, x, 3, None, r.handle),
                 lambda: pkv.kv_append_tokens(c, x, x, 7, 4096, r.handle)]:
        pkv.kv_testing_fail_launches(1)
        try:
            assert code(pkv, call) == "CUDA"
        finally:
            pkv.kv_testing_fail_launches(0)


def test_tensors_are_checked_before_the_call(pkv):
    import torch
    r = pkv.Rope(64)
    x, pos = torch.zeros(3, 2, 64, dtype=torch.bfloat16), torch.zeros(3, dtype=torch.int32)
    for a, p in [(x, pos), (x[0], pos), (x.double(), pos), (x, pos.long()), (x, pos[:2]),
                 (x.transpose(1, 2), pos), (x.permute(2, 1, 0), pos)]:
        with pytest.raises(ValueError):
            r.rotate(a, p)
    with pytest.raises(ValueError):
        r.rotate(x.float().requires_grad_(), pos, out=torch.empty(3, 2, 64))
    with pytest.raises(ValueError):
        pkv.PagedTokens(torch.zeros(4, 2, 16, 2, 64, dtype=torch.bfloat16), torch.zeros(1, 2, dtype=torch.int32),
                        torch.zeros(1, dtype=torch.int32))
    with pytest.raises(ValueError):
        pkv.PagedTokens(torch.zeros(4, 3, 16, 2, 64, dtype=torch.bfloat16), None, None)
    with pytest.raises(ValueError):
        pkv.PagedTokens(torch.zeros(4, 2, 16, 2, 64), None, None)


def test_counts_and_scales_at_the_edge_of_their_types(pkv):
    """Counts whose next row would not fit 31 bits, and scales that are finite but not in powers of two."""
    r, x, c, big = pkv.Rope(2), rows(pkv), tokens(pkv), 1 << 30
    for n, h in [(big + 1, 1), (2**31 - 1, 1), (1, big + 1), (1, 2**31 - 1)]:
        assert code(pkv, pkv.kv_rotate, r.handle, x, x, 4096, n, h, 2, 0) == "ARG"
    assert code(pkv, pkv.kv_append_tokens, c, x, x, 2**31 - 1, 4096) == "ARG"
    for scale in (3e38, -3e38):
        assert code(pkv, pkv.kv_decode, c, x, 2, scale, 0, 4096, 4096, big) == "ARG"
        assert code(pkv, pkv.kv_decode_append, c, x, x, x, 2, None, None, scale, 0, 4096, 4096, big) == "ARG"


# ---------------------------------------------------------------- frame plans
def test_plans_whose_tables_do_not_hold_are_refused(pkv):
    """kv_plan_check and PagedTokens.of_plan take a plan where its tokens are in the pool, stream by stream and block by block."""
    import torch
    caches = pkv.PagedKVCache.group(2, 40, 16, 2, 64, scale_frames=1, window=2, num_special=4, num_blocks=2)
    caches[0].pools[:] = [torch.zeros(40, 2, 16, 2, 64, dtype=torch.bfloat16)] * 2   # stand-ins: no call reaches them

    def frame(c, blocks=(0, 1)):
        for b in blocks:
            c.append_frame(b, None, None)
        c.evict_frames()

    def of_plan(plan, block, streams=None):   # refused for its state (KVError), or only then for not being on a GPU
        try:
            pkv.PagedTokens.of_plan(plan, block, streams)
        except pkv.KVError as e:
            return e.name
        except ValueError as e:
            assert "CUDA" in str(e)
            return "OK"

    for _ in range(4):
        frame(caches[0])
        frame(caches[1])
    plan = pkv.Plan(caches)
    assert [of_plan(plan, b) for b in (0, 1)] == ["OK", "OK"]
    frame(caches[1])                                    # its oldest page is another frame's by then
    assert of_plan(plan, 0) == of_plan(plan, 0, [1]) == "STALE_PLAN" and of_plan(plan, 0, [0]) == "OK"
    pkv.kv_plan_check(plan.handle, 0, 1)
    assert code(pkv, pkv.kv_plan_check, plan.handle, 1, 0) == "STALE_PLAN"
    caches[0].begin_frame()                             # a step's pages are taken, its blocks not written
    plan = pkv.Plan(caches)
    assert of_plan(plan, 0) == of_plan(plan, 1, [0]) == "NOT_APPENDED" and of_plan(plan, 0, [1]) == "OK"
    caches[0].append_frame(0, None, None)
    assert of_plan(plan, 0) == "OK" and of_plan(plan, 1) == "NOT_APPENDED"
    caches[0].append_frame(1, None, None)
    assert of_plan(plan, 1) == "OK"
    caches[1].defer_eviction()
    frame(caches[1])
    caches[1].rollback_last_frame()                     # what is left is written, with no step open
    assert of_plan(plan, 1, [1]) == "STALE_PLAN" and of_plan(pkv.Plan(caches), 1) == "OK"
    caches[1].reset()
    assert of_plan(plan, 1, [1]) == "STALE_PLAN"
    for args in ((None, 0, 0), (plan.handle, 2, 0), (plan.handle, -1, 0), (plan.handle, 0, 2), (plan.handle, 0, -1)):
        assert code(pkv, pkv.kv_plan_check, *args) == "ARG"


# ---------------------------------------------------------------- the binding's build
def test_the_binding_is_built_again_for_another_torch(pkv, monkeypatch, tmp_path):
    from paged_kv_cache_frame_b200 import build
    assert not build.binding_stale()
    for name, was in (("version", "1.0"), ("none", None)):
        at = tmp_path / name
        if was is not None:
            at.write_text(f"{was} {build._torch_and_python().split()[-1]}")
        monkeypatch.setattr(build, "BINDING_MADE_FOR", str(at))
        assert build.binding_stale()


# ---------------------------------------------------------------- index arithmetic
@pytest.mark.skipif(shutil.which("g++") is None, reason="needs g++")
def test_page_divisor(tmp_path):
    exe = tmp_path / "page_divisor"
    subprocess.run(["g++", "-std=c++17", "-O2", "-I", CSRC, os.path.join(HERE, "cpp", "page_divisor.cpp"),
                    "-o", str(exe)], check=True)
    r = subprocess.run([str(exe)], capture_output=True, text=True)
    assert r.returncode == 0 and r.stdout.startswith("ok "), r.stdout + r.stderr


@pytest.mark.skipif(shutil.which("g++") is None, reason="needs g++")
@pytest.mark.parametrize("name,headers", [("overlap", os.path.join(CSRC, "..", "binding")), ("decode_split", CSRC)])
def test_rules_that_the_kernels_and_the_binding_use(tmp_path, name, headers):
    exe = tmp_path / name
    subprocess.run(["g++", "-std=c++17", "-O2", "-I", headers, os.path.join(HERE, "cpp", name + ".cpp"), "-o", str(exe)], check=True)
    r = subprocess.run([str(exe)], capture_output=True, text=True)
    assert r.returncode == 0 and r.stdout.startswith("ok "), r.stdout + r.stderr


def find_seq(cu, n, t):
    """The kernel's search."""
    lo, hi = 0, n
    while lo < hi:
        mid = (lo + hi) // 2
        if cu[mid + 1] <= t:
            lo = mid + 1
        else:
            hi = mid
    return lo


def test_sequence_search():
    rng = random.Random(5)
    for n in (1, 2, 31, 32, 33, 64, 100, 1000, 1024, 1025, 5000):
        cu = [0]
        for _ in range(n):
            cu.append(cu[-1] + rng.choice([0, 0, 1, 3]))
        for t in sorted({0, cu[-1] - 1, cu[-1], cu[-1] + 5, *(rng.randrange(cu[-1] + 1) for _ in range(60))}):
            if t >= 0:
                assert find_seq(cu, n, t) == sum(c <= t for c in cu[1:])
    # out of order: any answer in range will do, the search ends and reads in range
    for _ in range(300):
        n = rng.randint(1, 3000)
        cu = [rng.randint(-5, 50) for _ in range(n + 1)]
        assert 0 <= find_seq(cu, n, rng.randint(0, 50)) <= n


JOIN, GROUP = 32, 16      # parts joined in one round, and neighbours joined first where there are more
PART, COST = 3, 2         # tiles a part holds at most, a sequence's own cost in the line


def split_pieces(tiles, ranks):
    """The pieces of every rank as the attention kernel splits them: sequence,
    rank, tiles, the sequence's first rank and its parts."""
    parts_of = lambda n: (n + PART - 1) // PART  # noqa: E731
    n_parts = sum(parts_of(n) for n in tiles)
    by_parts = n_parts <= ranks
    each, more = divmod(sum(n + COST for n in tiles if n), ranks)

    def rank_of(place):
        lower = more * (each + 1)
        return place // (each + 1) if place < lower else more + (place - lower) // each

    pieces = []
    for r in range(ranks):
        if by_parts:
            t, end = min(r, n_parts), min(r + 1, n_parts)
        else:
            t = r * each + min(r, more)
            end = t + each + (r < more)
        base, seq = 0, 0
        while t < end:
            while True:
                n = tiles[seq]
                size = parts_of(n) if by_parts else n + COST if n else 0
                if t - base < size:
                    break
                base += size
                seq += 1
            at = t - base
            if by_parts:
                t0, t1 = n * at // size, n * (at + 1) // size
                r0, parts = t - at, size
                t += 1
            else:
                took = min(end - t, size - at)
                t0, t1 = max(0, at - COST), max(0, at + took - COST)
                first = t - at
                r0 = r if t0 == 0 else rank_of(first + COST)
                parts = (r if t1 == n else rank_of(first + size - 1)) - r0 + 1
                t += took
            if t0 < t1:
                pieces.append((seq, r, t0, t1, r0, parts))
    return pieces


@pytest.mark.parametrize("seed", range(120))
def test_split_covers_every_tile_and_the_join_finds_the_parts(seed):
    """Every tile once; a sequence's parts in neighbouring ranks and slots no
    other part has; arrivals counted to the number that comes, on counters no
    two sequences (and no two units) share."""
    rng = random.Random(seed)
    seqs, ranks, units = rng.choice([1, 2, 7, 64, 300]), rng.choice([1, 4, 37, 296]), rng.choice([1, 3])
    most = rng.choice([3, 20, 400, 9000])
    tiles = [rng.choice([0, 1, 2, 5, rng.randint(0, most)]) for _ in range(seqs)]
    pieces = split_pieces(tiles, ranks)
    assert set(p[0] for p in pieces) == {s for s in range(seqs) if tiles[s]}
    by_seq, slots, first, second = {}, set(), {}, {}
    slot = lambda r0, p, u: 2 * ((r0 + p) * units + u) + (p == 0)  # noqa: E731
    for seq, r, t0, t1, r0, n in pieces:
        by_seq.setdefault(seq, []).append((t0, t1, r, r0, n))
        assert n == 1 or ranks > 1
        for u in range(units if n > 1 else 0):
            here = slot(r0, r - r0, u)
            assert here < 2 * ranks * units and here not in slots
            slots.add(here)
            two, me = n > JOIN, r - r0
            g0 = me // GROUP * GROUP if two else 0
            first.setdefault(slot(r0, g0, u), []).append((seq, u, min(GROUP, n - g0) if two else n))
            if two and me == g0:
                second.setdefault(slot(r0, 0, u), []).append((seq, u, (n + GROUP - 1) // GROUP))
    for counters in (first, second):
        for arrivals in counters.values():
            assert len(set(arrivals)) == 1 and len(arrivals) == arrivals[0][2] <= JOIN
    for seq, p in by_seq.items():
        p.sort()
        assert p[0][0] == 0 and p[-1][1] == tiles[seq] and all(a[1] == b[0] for a, b in zip(p, p[1:]))
        assert [x[2:] for x in p] == [(p[0][3] + i, p[0][3], len(p)) for i in range(len(p))]
