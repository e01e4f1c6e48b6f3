"""Cases for the token operators: rotary positions, appending tokens to a paged
pool, attention of one new token over it, and the decode step that does all
three in one call.

Pools are [max_pages, 2 (K/V), page_size, kv heads, head_dim], as everywhere in
this package. Sequence s keeps its token j in row j % page_size of page
tables[s][j // page_size]; lens[s] counts its tokens, the new ones included.

Each case has a plain form (`own` false: products, sums, exponentials and
indexing in 32 bits, angles in 64) and the package's call (`own` true).
"""
import math
import random

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}


def _rope(rot, layout="half", scaling="none", factor=1.0, context=0, base=10000.0):
    return {"rot": rot, "layout": layout, "scaling": scaling, "factor": factor, "context": context, "base": base}


def listed():
    return [
        # One new token of each of 8 streams: the queries of a decode step, the
        # smallest call, all latency.
        {"name": "rotate-token", "kind": "rotate", "dtype": "bf16", "tokens": 8, "heads": 16, "head_dim": 64,
         "far": 20000, **_rope(64)},
        # The queries and keys of a long prompt, next to each other as the
        # fused projection leaves them, far past the trained context.
        {"name": "rotate-prompt", "kind": "rotate", "dtype": "bf16", "tokens": 8192, "heads": 40, "head_dim": 128,
         "far": 131072, **_rope(128, "half", "yarn", 4.0, 32768)},
        # A training step: the rotation and its gradient, in 32 bits, half of
        # the head, neighbouring pairs, an odd number of rows.
        {"name": "rotate-train", "kind": "train", "dtype": "fp32", "tokens": 4095, "heads": 24, "head_dim": 128,
         "far": 4096, **_rope(64, "interleaved", "linear", 2.0)},
        # One new token of each of 64 sequences, into pages of a 224x224 frame.
        {"name": "append-step", "kind": "append", "dtype": "bf16", "seqs": 64, "kv_heads": 16, "head_dim": 64,
         "page": 256, "new_most": 1, "prior_most": 2000, **_rope(64)},
        # Prompts of unequal length (some pages already begun), as a serving
        # program batches them.
        {"name": "append-prompts", "kind": "append", "dtype": "fp16", "seqs": 9, "kv_heads": 8, "head_dim": 128,
         "page": 64, "new_most": 5011, "prior_most": 700, **_rope(128, "half", "ntk", 8.0)},
        # One token against a short cache: the smallest attention call.
        {"name": "decode-short", "kind": "decode", "dtype": "bf16", "seqs": 1, "kv_heads": 16, "group": 1,
         "head_dim": 64, "page": 256, "least": 300, "most": 300, "empty": False, "window": 0},
        # One token against everything a 224x224 stream of 320 frames shows:
        # 72 frames of 256 patch tokens and 320 frames of 6 special ones.
        {"name": "decode-stream", "kind": "decode", "dtype": "bf16", "seqs": 1, "kv_heads": 16, "group": 1,
         "head_dim": 64, "page": 256, "least": 20352, "most": 20352, "empty": False, "window": 0},
        # Four 518x378 streams of 1000 frames: the largest call, odd pages.
        {"name": "decode-streams-large", "kind": "decode", "dtype": "bf16", "seqs": 4, "kv_heads": 16, "group": 1,
         "head_dim": 64, "page": 999, "least": 77928, "most": 77928, "empty": False, "window": 0},
        # A serving batch of unequal lengths with shared heads and one unused row.
        {"name": "decode-batch", "kind": "decode", "dtype": "fp16", "seqs": 64, "kv_heads": 8, "group": 4,
         "head_dim": 128, "page": 16, "least": 1, "most": 8192, "empty": True, "window": 0},
        # One very long sequence: few rows, all of the work along the cache.
        {"name": "decode-long", "kind": "decode", "dtype": "bf16", "seqs": 1, "kv_heads": 4, "group": 8,
         "head_dim": 128, "page": 64, "least": 262111, "most": 262111, "empty": False, "window": 0},
        # The whole decode step of two short sequences.
        {"name": "step-short", "kind": "step", "dtype": "bf16", "seqs": 2, "kv_heads": 8, "group": 2,
         "head_dim": 128, "page": 256, "least": 500, "most": 1000, "empty": False, "window": 0, **_rope(128)},
        # The whole decode step of a padded batch with a sliding window.
        {"name": "step-batch", "kind": "step", "dtype": "bf16", "seqs": 128, "kv_heads": 4, "group": 7,
         "head_dim": 64, "page": 17, "least": 1, "most": 4100, "empty": True, "window": 1500,
         **_rope(48, "interleaved", "yarn", 8.0, 1024)},
    ]


def _log_int(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def _draw_rope(rng, head_dim):
    rot = head_dim if rng.random() < 0.5 else 2 * rng.randint(1, head_dim // 2)
    scaling = rng.choice(["none", "linear", "ntk", "yarn"])
    factor = 1.0 if scaling == "none" else round(rng.uniform(1.5, 32.0), 2)
    context = rng.choice([512, 2048, 8192, 32768]) if scaling == "yarn" else 0
    return _rope(rot, rng.choice(["half", "interleaved"]), scaling, factor, context, rng.choice([10000.0, 500000.0]))


def draw(rng):
    kind = rng.choice(["rotate", "train", "append", "decode", "decode", "decode", "step", "step"])
    if kind in ("rotate", "train"):
        d = rng.choice([64, 80, 96, 128, 256])
        tokens, heads = _log_int(rng, 1, 8192), _log_int(rng, 1, 40)
        if tokens * heads * d > 8192 * 40 * 128:
            tokens = 8192 * 40 * 128 // (heads * d)
        if kind == "train":
            tokens = min(tokens, max(1, 4095 * 24 * 128 // (heads * d)))
        return {"kind": kind, "dtype": rng.choice(["bf16", "fp16", "fp32"]), "tokens": tokens, "heads": heads,
                "head_dim": d, "far": rng.choice([4096, 131072, 1000000]), **_draw_rope(rng, d)}
    case = {"kind": kind, "dtype": rng.choice(["bf16", "fp16"]), "kv_heads": rng.choice([1, 2, 3, 4, 8, 16]),
            "head_dim": rng.choice([64, 128]), "page": rng.choice([16, 64, 256, 999, rng.randint(1, 400)])}
    if kind == "append":
        seqs = _log_int(rng, 1, 256)
        new = _log_int(rng, 1, max(1, 20000 // seqs))
        return {**case, "seqs": seqs, "new_most": new, "prior_most": _log_int(rng, 1, 900),
                **_draw_rope(rng, case["head_dim"])}
    seqs = _log_int(rng, 1, 128)
    row = case["kv_heads"] * case["head_dim"]
    room = (4 * 77928 * 16 * 64 if kind == "decode" else 128 * 4100 * 4 * 64) // (seqs * row)
    group = rng.choice([1, 2, 3, 4, 5, 7, 8, 16])
    room = min(room, 8 * 262111 * 4 * 128 // (seqs * row * group))
    most = _log_int(rng, 1, max(1, min(262144 if kind == "decode" else 16384, room)))
    case.update({"seqs": seqs, "group": group, "least": _log_int(rng, 1, most),
                 "most": most, "empty": seqs > 1 and rng.random() < 0.3,
                 "window": _log_int(rng, 1, most) if rng.random() < 0.3 else 0})
    return case if kind == "decode" else {**case, **_draw_rope(rng, case["head_dim"])}


def _lens(case):
    """Tokens of each sequence, the new ones included."""
    rng = random.Random(1000003 * case["seqs"] + case["page"])
    if case["kind"] == "append":
        new = [_log_int(rng, 1, case["new_most"]) for _ in range(case["seqs"])]
        new[0] = case["new_most"]
        return [n + rng.randint(0, case["prior_most"]) for n in new], new
    lens = [rng.randint(case["least"], case["most"]) for _ in range(case["seqs"])]
    lens[0] = case["most"]
    if case["empty"]:
        lens[-1] = 0
    return lens, [1] * case["seqs"]


def _randn(shape, dtype, gen):
    return torch.randn(shape, generator=gen, device="cuda", dtype=torch.float32).to(dtype)


def _frequencies(case):
    """Rotation of each pair in radians a position, and the amplitude of the rotated values."""
    i = torch.arange(case["rot"] // 2, device="cuda", dtype=torch.float64)
    freq = case["base"] ** (-2.0 * i / case["rot"])
    if case["scaling"] == "linear":
        return freq / case["factor"], 1.0
    if case["scaling"] == "ntk":
        return freq * case["factor"] ** (-2.0 * i / max(1, case["rot"] - 2)), 1.0
    if case["scaling"] == "yarn":
        turns = case["context"] * freq / (2 * math.pi)
        keep = ((turns - 1.0) / (32.0 - 1.0)).clamp(0, 1)
        return freq * (keep + (1 - keep) / case["factor"]), 0.1 * math.log(case["factor"]) + 1.0
    return freq, 1.0


def _handle(case):
    import paged_kv_cache_frame_b200 as pkv
    return pkv.Rope(case["rot"], layout=case["layout"], base=case["base"], scaling=case["scaling"],
                    factor=case["factor"], original_context=case["context"])


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    dtype = DTYPES[case["dtype"]]
    st = {"case": case}
    if "rot" in case:
        st["freq"], st["amplitude"] = _frequencies(case)
        if own:
            st["rope"] = _handle(case)
    if case["kind"] in ("rotate", "train"):
        n, h, d = case["tokens"], case["heads"], case["head_dim"]
        st["x"] = _randn((n, h, d), dtype, gen)
        first = torch.randint(0, case["far"], (1,), generator=gen, device="cuda")
        st["positions"] = (first + torch.arange(n, device="cuda")).to(torch.int32)
        if case["kind"] == "train":
            st["x"].requires_grad_()
            st["dy"] = _randn((n, h, d), dtype, gen)
        return st
    lens, new = _lens(case)
    hkv, d, ps, s = case["kv_heads"], case["head_dim"], case["page"], case["seqs"]
    pages = [-(-n // ps) for n in lens]
    width = max(pages)
    pool_pages = sum(pages) + 3
    order = torch.randperm(pool_pages, generator=gen, device="cuda").to(torch.int32)
    rows, at = [], 0
    for n in pages:
        rows.append(torch.nn.functional.pad(order[at:at + n], (0, width - n)))
        at += n
    st["tables"] = torch.stack(rows)
    st["spare"] = order[-1].long()
    st["lens"] = torch.tensor(lens, dtype=torch.int32, device="cuda")
    st["pool"] = torch.empty((pool_pages, 2, ps, hkv, d), dtype=dtype, device="cuda")
    flat = st["pool"].view(-1)
    for a in range(0, flat.numel(), 1 << 28):
        flat[a:a + (1 << 28)] = _randn((min(1 << 28, flat.numel() - a),), dtype, gen)
    st["longest"] = width * ps
    if case["kind"] == "append":
        st["cu_new"] = torch.tensor([0] + new, device="cuda").cumsum(0).to(torch.int32) if case["new_most"] > 1 else None
    if case["kind"] in ("append", "step"):
        st["k"] = _randn((sum(new), hkv, d), dtype, gen)
        st["v"] = _randn((sum(new), hkv, d), dtype, gen)
    if case["kind"] in ("decode", "step"):
        st["q"] = _randn((s, hkv * case["group"], d), dtype, gen)
    if own:
        import paged_kv_cache_frame_b200 as pkv
        st["cache"] = pkv.PagedTokens(st["pool"], st["tables"], st["lens"])
    return st


# ---------------------------------------------------------------- plain forms
def _turn(x, positions, st, sign=1.0):
    """x [n, heads, head_dim] in 32 bits, its first `rot` values rotated; 32 bits out."""
    case = st["case"]
    rot = case["rot"]
    angle = positions.double()[:, None] * st["freq"]
    cos = (angle.cos() * st["amplitude"]).float()[:, None]
    sin = (angle.sin() * (st["amplitude"] * sign)).float()[:, None]
    x = x.float()
    if case["layout"] == "half":
        a, b = x[..., :rot // 2], x[..., rot // 2:rot]
        r = torch.cat([a * cos - b * sin, b * cos + a * sin], -1)
    else:
        a, b = x[..., 0:rot:2], x[..., 1:rot:2]
        r = torch.stack([a * cos - b * sin, b * cos + a * sin], -1).flatten(-2)
    return torch.cat([r, x[..., rot:]], -1)


def _slots(st, seq, index):
    """Page and row of token `index` of sequence `seq`."""
    ps = st["case"]["page"]
    return st["tables"][seq, index // ps].long(), index % ps


def _append(st):
    """The new tokens into the pool: keys rotated, values as they are."""
    lens = st["lens"].long()
    n = st["k"].shape[0]
    t = torch.arange(n, device="cuda")
    if st.get("cu_new") is None:
        seq, index = t, lens - 1
    else:
        cu = st["cu_new"].long()
        seq = torch.searchsorted(cu[1:], t, right=True)
        index = lens[seq] - (cu[seq + 1] - t)
    k = _turn(st["k"], index, st).to(st["pool"].dtype)
    # an unused row of the batch keeps what a page of no sequence holds
    live = (index >= 0)[:, None, None]
    page, row = _slots(st, seq, index.clamp_min(0))
    page = torch.where(index >= 0, page, st["spare"])
    st["pool"][page, 0, row] = torch.where(live, k, st["pool"][page, 0, row])
    st["pool"][page, 1, row] = torch.where(live, st["v"], st["pool"][page, 1, row])


def _attend(st, q):
    """q [seqs, q heads, head_dim] in 32 bits against each sequence's tokens."""
    case = st["case"]
    s, hkv, d = case["seqs"], case["kv_heads"], case["head_dim"]
    kv = st["pool"][st["tables"].long()]                              # [seqs, pages, 2, page, kv heads, head_dim]
    k = kv[:, :, 0].reshape(s, -1, hkv, d).permute(0, 2, 3, 1).float()
    scores = torch.matmul(q.view(s, hkv, -1, d), k) / math.sqrt(d)    # [seqs, kv heads, group, tokens]
    del k
    j = torch.arange(scores.shape[-1], device="cuda")
    seen = j < st["lens"][:, None]
    if case["window"]:
        seen = seen & (j >= st["lens"][:, None] - case["window"])
    seen = seen[:, None, None]
    scores = scores.masked_fill(~seen, -math.inf)
    top = scores.amax(-1, keepdim=True)
    p = torch.where(seen, (scores - top).exp(), torch.zeros_like(scores))
    v = kv[:, :, 1].reshape(s, -1, hkv, d).permute(0, 2, 1, 3).float()
    v = torch.where(seen[:, :, 0, :, None], v, torch.zeros_like(v))
    out = torch.matmul(p, v) / p.sum(-1, keepdim=True).clamp_min(1e-30)
    return out.view(s, -1, d).to(st["pool"].dtype)


def run(st):
    case = st["case"]
    kind = case["kind"]
    if kind == "rotate":
        if own:
            return st["rope"].rotate(st["x"], st["positions"])
        return _turn(st["x"], st["positions"], st).to(st["x"].dtype)
    if kind == "train":
        if own:
            y = st["rope"].rotate(st["x"], st["positions"])
            return y.detach(), torch.autograd.grad(y, st["x"], st["dy"])[0]
        with torch.no_grad():
            y = _turn(st["x"], st["positions"], st).to(st["x"].dtype)
            return y, _turn(st["dy"], st["positions"], st, -1.0).to(st["x"].dtype)
    if kind == "append":
        if own:
            st["cache"].append(st["k"], st["v"], cu_new=st["cu_new"], rope=st["rope"])
        else:
            _append(st)
        return st["pool"]
    if kind == "decode":
        if own:
            return st["cache"].decode(st["q"], window=case["window"])
        return _attend(st, st["q"].float())
    if own:
        return st["cache"].decode_append(st["k"], st["v"], st["q"], rope=st["rope"], window=case["window"]), st["pool"]
    _append(st)
    return _attend(st, _turn(st["q"], st["lens"] - 1, st)), st["pool"]


# ---------------------------------------------------------------- work, exact values
def work(case):
    size = 4 if case["dtype"] == "fp32" else 2
    if case["kind"] in ("rotate", "train"):
        n, h, d = case["tokens"], case["heads"], case["head_dim"]
        passes = 2 if case["kind"] == "train" else 1
        return {"bytes": passes * (2 * n * h * d * size + 4 * n), "flops": passes * 3 * n * h * case["rot"]}
    lens, new = _lens(case)
    if case["kind"] != "append":
        new = [min(1, n) for n in lens]
    row = case["kv_heads"] * case["head_dim"]
    total = {"bytes": 0, "flops": 0}
    if case["kind"] in ("append", "step"):
        # k and v read and written once, and the tables' entries of the pages touched
        total["bytes"] += 4 * sum(new) * row * size + 4 * len(new)
        total["flops"] += 3 * sum(new) * case["kv_heads"] * case["rot"]
    if case["kind"] in ("decode", "step"):
        seen = sum(min(n, case["window"]) if case["window"] else n for n in lens)
        old = seen - (sum(new) if case["kind"] == "step" else 0)
        q = case["seqs"] * row * case["group"]
        total["bytes"] += 2 * old * row * size + 2 * q * size + 4 * len(lens) + 4 * (seen // case["page"] + 1)
        total["flops"] += 4 * seen * row * case["group"]
    return total


def _exact_turn(x, positions, case, sign=1.0):
    """The rotation pair by pair, as complex numbers in 64 bits."""
    rot, s = case["rot"], case["factor"]
    amplitude, theta = 1.0, []
    for i in range(rot // 2):
        f = case["base"] ** (-2.0 * i / rot)
        if case["scaling"] == "linear":
            f /= s
        elif case["scaling"] == "ntk" and i:
            f /= s ** (2.0 * i / (rot - 2))
        elif case["scaling"] == "yarn":
            keep = min(1.0, max(0.0, (case["context"] * f / (2 * math.pi) - 1.0) / 31.0))
            f = keep * f + (1 - keep) * f / s
        theta.append(f)
    if case["scaling"] == "yarn":
        amplitude = 1.0 + 0.1 * math.log(s)
    x = x.detach().double().clone()
    angle = sign * positions.double().outer(torch.tensor(theta, dtype=torch.float64, device=x.device))
    turn = torch.polar(torch.full_like(angle, amplitude), angle)[:, None, :]
    if case["layout"] == "half":
        z = torch.complex(x[..., :rot // 2], x[..., rot // 2:rot]) * turn
        x[..., :rot // 2], x[..., rot // 2:rot] = z.real, z.imag
    else:
        x[..., :rot] = torch.view_as_real(torch.view_as_complex(x[..., :rot].unflatten(-1, (-1, 2)).contiguous()) * turn).flatten(-2)
    return x


def exact(case, seed):
    st = prepare(case, seed)
    if case["kind"] == "rotate":
        return _exact_turn(st["x"], st["positions"], case)
    if case["kind"] == "train":
        return _exact_turn(st["x"], st["positions"], case), _exact_turn(st["dy"], st["positions"], case, -1.0)
    lens, new = _lens(case)
    ps, d, g = case["page"], case["head_dim"], case.get("group", 1)
    pool = st["pool"].double() if case["kind"] != "decode" else st["pool"]
    tables = st["tables"].tolist()
    if case["kind"] in ("append", "step"):
        at = 0
        for s, (n, m) in enumerate(zip(lens, new)):
            if n:
                index = torch.arange(n - m, n)
                page = torch.tensor([tables[s][j // ps] for j in index.tolist()], device="cuda")
                row = (index % ps).cuda()
                pool[page, 0, row] = _exact_turn(st["k"][at:at + m], index.cuda(), case)
                pool[page, 1, row] = st["v"][at:at + m].double()
            at += m
    if case["kind"] == "append":
        return pool
    q = st["q"].double()
    if case["kind"] == "step":
        q = _exact_turn(q, st["lens"] - 1, case)
    out = torch.zeros_like(q)
    for s, n in enumerate(lens):
        if not n:
            continue
        first = max(0, n - case["window"]) if case["window"] else 0
        pages = torch.tensor(tables[s][:-(-n // ps)], device="cuda")
        for h in range(case["kv_heads"]):
            k = pool[pages, 0, :, h].reshape(-1, d)[first:n].double()
            v = pool[pages, 1, :, h].reshape(-1, d)[first:n].double()
            out[s, h * g:(h + 1) * g] = torch.softmax(q[s, h * g:(h + 1) * g] @ k.T * d ** -0.5, -1) @ v
    return out if case["kind"] == "decode" else (out, pool)
