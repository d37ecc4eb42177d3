"""Cases of the drafted-token operators: rotary positions, appending rotated keys and values to
the segment cache, attention for trees of drafted tokens, and moving accepted rows.

``listed()`` gives the named cases, ``draw(rng)`` one more of the same ranges.  ``prepare`` makes
a case's inputs on the GPU, ``run`` computes one pass: the operators' plain form in elementary
torch operations, or, where ``own`` is true, the library's calls.  ``exact`` computes the same
values from the operators' definitions in 64 bits.

Shapes are those of this repository's workloads: 64 / 8 heads of 128, with 8 / 1 and 16 / 2 heads
of 64 and 32 / 32 heads of 128 beside them; contexts of 1 thousand to 131 thousand keys in
segments of a shared pool; batches of 1 to 128 requests.
"""
import math

import numpy as np
import torch

own = False

DEV = "cuda"


# ------------------------------------------------------------------------------- cases
def _rope(name, tokens, heads=64, head_dim=128, rotary=128, interleaved=False, scaling="none",
          factor=1.0, base=10000.0, span=4096, backward=False):
    return dict(name=name, op="rope", tokens=tokens, heads=heads, head_dim=head_dim, rotary=rotary,
                interleaved=interleaved, scaling=scaling, factor=factor, base=base, span=span,
                backward=backward)


def _append(name, tokens, q_heads=64, kv_heads=8, head_dim=128, rotary=128, interleaved=False,
            scaling="none", factor=1.0, base=10000.0, span=32768, fp8=False):
    return dict(name=name, op="append", tokens=tokens, q_heads=q_heads, kv_heads=kv_heads,
                head_dim=head_dim, rotary=rotary, interleaved=interleaved, scaling=scaling,
                factor=factor, base=base, span=span, fp8=fp8)


def _tree(name, batch, draft_min, draft_max, prior_min, prior_max, q_heads=64, kv_heads=8,
          head_dim=128, segments=4, fp8=False, form="tree"):
    return dict(name=name, op="tree", batch=batch, draft_min=draft_min, draft_max=draft_max,
                prior_min=prior_min, prior_max=prior_max, q_heads=q_heads, kv_heads=kv_heads,
                head_dim=head_dim, segments=segments, fp8=fp8, form=form)


def _move(name, batch, draft, accept_max, kv_heads=8, head_dim=128, fp8=False):
    return dict(name=name, op="move", batch=batch, draft=draft, accept_max=accept_max,
                kv_heads=kv_heads, head_dim=head_dim, fp8=fp8)


def listed():
    return [
        # the queries of one decoded token: the smallest call, all latency
        _rope("rope one token", 1),
        # a prefill chunk with half of each head rotated, adjacent pairs
        _rope("rope chunk, half the head", 2048, rotary=64, interleaved=True),
        # gradients of a long training sequence's queries, positions scaled past the first 8192
        _rope("rope long, backward", 16381, scaling="yarn", factor=32.0, base=500000.0,
              span=262144, backward=True),
        # the new tokens of a decode step of 128 requests
        _append("append 128 decodes", 128),
        # a prefill chunk into an E4M3 cache, long-context positions
        _append("append chunk, E4M3", 2047, scaling="wavelength", factor=8.0, base=500000.0,
                span=131072, fp8=True),
        # many prompts at once
        _append("append 16k tokens", 16384),
        # one conversation, a small tree of drafts: latency
        _tree("tree 1 x 8 over 1k", 1, 8, 8, 1021, 1021),
        # a serving batch: trees of different sizes over contexts of different lengths
        _tree("tree 32 x 4-32 over 1k-8k", 32, 4, 32, 1024, 8192),
        # long contexts, the drafts read the whole cache once
        _tree("tree 8 x 16 over 131k", 8, 16, 16, 131072, 131072, segments=16),
        # wide trees over an E4M3 cache
        _tree("tree 64 x 1-64 over 0-8k, E4M3", 64, 1, 64, 0, 8192, segments=8, fp8=True),
        # what one request accepted
        _move("move 1 x 5", 1, 16, 5),
        # what a batch of 128 accepted
        _move("move 128 x 1-8", 128, 32, 8),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["rope", "append", "tree", "tree", "move"])
    heads, kv, d = rng.choice([(64, 8, 128), (32, 32, 128), (16, 2, 64), (8, 1, 64)])
    rot = dict(rotary=rng.choice([d, d, d // 2, d // 4]), interleaved=rng.random() < 0.5,
               scaling=rng.choice(["none", "linear", "ntk", "yarn", "wavelength"]),
               factor=rng.choice([2.0, 4.0, 8.0, 32.0]), base=rng.choice([10000.0, 500000.0]),
               span=_log_int(rng, 512, 1 << 20))
    if op == "rope":
        c = _rope("", _log_int(rng, 1, 16000), heads, d, backward=rng.random() < 0.3, **rot)
    elif op == "append":
        c = _append("", _log_int(rng, 1, 16000), heads, kv, d, fp8=rng.random() < 0.4, **rot)
    elif op == "move":
        batch = _log_int(rng, 1, 128)
        c = _move("", batch, rng.randint(8, 64), rng.randint(1, 8), kv, d, rng.random() < 0.4)
    else:
        draft = _log_int(rng, 1, 64)
        prior = _log_int(rng, 64, 131072)
        # no more of the cache, and no more scores, than the largest listed case has
        keys = prior + draft
        most = min((1 << 30) // (kv * d * keys), (1 << 30) // (heads * draft * keys), 64)
        batch = _log_int(rng, 1, max(1, most))
        c = _tree("", batch, rng.randint(1, draft), draft, rng.randint(0, prior), prior, heads, kv,
                  d, rng.randint(1, 16), rng.random() < 0.4, rng.choice(["tree", "chain", "mask"]))
    del c["name"]
    return c


def _spread(n, lo, hi):
    """n lengths from lo to hi, in no order; the same for every seed."""
    if n == 1:
        return [hi]
    return [lo + ((hi - lo) * ((k * 7919) % n) + (n - 1) // 2) // (n - 1) for k in range(n)]


def _lengths(case):
    draft = _spread(case["batch"], case["draft_min"], case["draft_max"])
    prior = _spread(case["batch"], case["prior_min"], case["prior_max"])[::-1]
    return draft, prior


def work(case):
    d = case["head_dim"]
    if case["op"] == "rope":
        n, h = case["tokens"], case["heads"]
        return {"bytes": 4 * n * h * d + 4 * n, "flops": 3 * n * h * case["rotary"]}
    if case["op"] == "append":
        n, hq, hk = case["tokens"], case["q_heads"], case["kv_heads"]
        cache = 2 * n * hk * d * (1 if case["fp8"] else 2)
        return {"bytes": 4 * n * hq * d + 4 * n * hk * d + cache + 8 * n,
                "flops": 3 * n * (hq + hk) * case["rotary"]}
    if case["op"] == "move":
        rows = sum(_spread(case["batch"], 1, case["accept_max"]))
        elem = 1 if case["fp8"] else 2
        return {"bytes": 4 * rows * case["kv_heads"] * d * elem + 8 * rows, "flops": 0}
    draft, prior = _lengths(case)
    hq, hk, elem = case["q_heads"], case["kv_heads"], 1 if case["fp8"] else 2
    keys = sum(draft) + sum(prior)
    # the drafted tokens' own keys count at what a chain would see; trees see fewer
    seen = sum(t * p + t * (t + 1) // 2 for t, p in zip(draft, prior))
    return {"bytes": 2 * keys * hk * d * elem + 4 * sum(draft) * hq * d + 4 * sum(draft) * hq,
            "flops": 4 * d * hq * seen}


# ------------------------------------------------------------------------------- inputs
YARN_LOW, YARN_HIGH = 1.0, 32.0      # turns over the original length where the ramp ends
WAVE_LOW, WAVE_HIGH = 1.0, 4.0       # original length over wavelength where the blend ends
ORIGINAL = 8192


def _inv_freq(case):
    """Radians per position of each pair (64 bits, numpy) and the factor on cos and sin."""
    r, base, s, f = case["rotary"], case["base"], case["scaling"], case["factor"]
    if s == "ntk" and r > 2:
        base = base * f ** (r / (r - 2))
    inv = base ** (-np.arange(0, r, 2, dtype=np.float64) / r)
    if s == "linear":
        inv = inv / f
    elif s == "yarn":
        pair = lambda turns: r * math.log(ORIGINAL / (turns * 2 * math.pi)) / (2 * math.log(base))
        lo = max(math.floor(pair(YARN_HIGH)), 0)
        hi = min(math.ceil(pair(YARN_LOW)), r - 1)
        ramp = np.clip((np.arange(r // 2) - lo) / max(hi - lo, 1e-3), 0, 1)
        inv = inv * (1 - ramp) + inv / f * ramp
        return inv, 0.1 * math.log(f) + 1.0
    elif s == "wavelength":
        turns = ORIGINAL * inv / (2 * math.pi)
        keep = np.clip((turns - WAVE_LOW) / (WAVE_HIGH - WAVE_LOW), 0, 1)
        inv = inv * keep + inv / f * (1 - keep)
    return inv, 1.0


def _plan(case):
    import segmented_kv_cache_b200 as sa
    s, kw = case["scaling"], dict(factor=case["factor"])
    if s == "yarn":
        kw.update(original_len=ORIGINAL, low=YARN_LOW, high=YARN_HIGH)
    elif s == "wavelength":
        kw.update(original_len=ORIGINAL, low=WAVE_LOW, high=WAVE_HIGH)
    scaling = None if s == "none" else sa.RopeScaling(s, **kw)
    return sa.seg_attn_rope_plan(case["rotary"], interleaved=case["interleaved"],
                                 base=case["base"], scaling=scaling)


def _normal(gen, *shape):
    return torch.randn(*shape, generator=gen, device=DEV, dtype=torch.float32).to(torch.bfloat16)


def _pool(gen, slots, heads, d, fp8):
    """A cache in use: every slot holds some request's values (E4M3 codes as bytes)."""
    x = torch.empty(slots, heads, d, dtype=torch.uint8 if fp8 else torch.bfloat16, device=DEV)
    for at in range(0, slots, 1 << 17):
        part = torch.randn(min(1 << 17, slots - at), heads, d, generator=gen, device=DEV)
        x[at:at + (1 << 17)] = ((part * 16).to(torch.float8_e4m3fn).view(torch.uint8) if fp8
                                else part.to(torch.bfloat16))
    return x


def _scales(heads):
    """Per-head scales of an E4M3 cache of values near N(0, 1)."""
    return (1 / 16 + torch.arange(heads, device=DEV, dtype=torch.float32) / 1024)


def _positions(rng, n, span):
    """Runs of positions of several requests, the last of them at the end of the span."""
    runs = max(1, min(n, 8))
    cut = np.sort(rng.randint(0, n + 1, runs - 1))
    pos = np.concatenate([rng.randint(0, span) + np.arange(b - a) for a, b in
                          zip(np.r_[0, cut], np.r_[cut, n])])
    pos[-1] = span - 1
    return torch.from_numpy(pos.astype(np.int32)).to(DEV)


def _place(rng, segments):
    """Pool slots for a list of (owner, length) runs, in an order of their own, with gaps."""
    start, at = [0] * len(segments), 0
    for i in rng.permutation(len(segments)):
        at += rng.randint(0, 9)
        start[i] = at
        at += segments[i][1]
    return start, sum(x for _, x in segments) + 9 * len(segments) + 9   # the same for every seed


def _parents(rng, n, form):
    """Parent of each drafted token (-1: the last cached token), parents before children."""
    if form == "chain":
        return [i - 1 for i in range(n)]
    # a few candidates at every depth, the first of them extended most
    return [-1 if i == 0 else int(i - 1 - min(i - 1, rng.randint(0, 4) * rng.randint(0, 3)))
            for i in range(n)]


def _ancestors(parents):
    n = len(parents)
    m = np.zeros((n, n), dtype=bool)
    for i, p in enumerate(parents):
        if p >= 0:
            m[i] = m[p]
        m[i, i] = True
    return m


def prepare(case, seed):
    gen = torch.Generator(device=DEV).manual_seed(seed)
    rng = np.random.RandomState(seed % (1 << 31))
    s = dict(case=case)
    if case["op"] in ("rope", "append"):
        n, d = case["tokens"], case["head_dim"]
        s["positions"] = _positions(rng, n, case["span"])
        inv, s["amp"] = _inv_freq(case)
        s["inv_freq"] = torch.from_numpy(inv).to(DEV)
        if own:
            s["rope"] = _plan(case)
    if case["op"] == "rope":
        s["x"] = _normal(gen, n, case["heads"], d)
        s["out"] = torch.empty_like(s["x"])
    elif case["op"] == "append":
        hq, hk = case["q_heads"], case["kv_heads"]
        # one projection's output: queries, keys and values of a token side by side
        qkv = _normal(gen, n, hq + 2 * hk, d)
        s["q"], s["k"], s["v"] = qkv[:, :hq], qkv[:, hq:hq + hk], qkv[:, hq + hk:]
        s["q_out"] = torch.empty(n, hq, d, dtype=torch.bfloat16, device=DEV)
        runs = np.array_split(np.arange(n), min(n, 16))
        start, slots = _place(rng, [(i, len(r)) for i, r in enumerate(runs)])
        at = np.concatenate([st + np.arange(len(r)) for st, r in zip(start, runs)])
        s["slots"] = torch.from_numpy(at.astype(np.int32)).to(DEV)
        s["k_pool"] = _pool(gen, slots, hk, d, case["fp8"])
        s["v_pool"] = _pool(gen, slots, hk, d, case["fp8"])
        s["k_scale"], s["v_scale"] = _scales(hk), _scales(hk) * 1.5
    elif case["op"] == "move":
        b, t = case["batch"], case["draft"]
        rows = _spread(b, 1, case["accept_max"])
        start, slots = _place(rng, [(r, t) for r in range(b)] + [(r, k) for r, k in enumerate(rows)])
        src, dst, offsets = [], [], [0]
        for r, k in enumerate(rows):
            # the accepted path: drafted tokens in increasing order, to the request's own run
            src.append(start[r] + np.sort(rng.permutation(t)[:min(k, t)]))
            dst.append(start[b + r] + np.arange(min(k, t)))
            offsets.append(offsets[-1] + min(k, t))
        i32 = lambda x: torch.from_numpy(np.asarray(x, dtype=np.int32)).to(DEV)
        s["src"], s["dst"], s["offsets"] = i32(np.concatenate(src)), i32(np.concatenate(dst)), i32(offsets)
        s["k_pool"] = _pool(gen, slots, case["kv_heads"], case["head_dim"], case["fp8"])
        s["v_pool"] = _pool(gen, slots, case["kv_heads"], case["head_dim"], case["fp8"])
    else:
        _prepare_tree(case, s, gen, rng)
    return s


def _prepare_tree(case, s, gen, rng):
    draft, prior = _lengths(case)
    b, hq, hk, d = case["batch"], case["q_heads"], case["kv_heads"], case["head_dim"]
    runs, owner = [], []
    for r in range(b):
        # the cached tokens in a few runs, the drafted ones in one of their own
        cuts = np.sort(rng.randint(0, prior[r] + 1, rng.randint(1, case["segments"] + 1) - 1))
        lens = [int(x) for x in np.diff(np.r_[0, cuts, prior[r]]) if x > 0]
        runs += [(r, x) for x in lens] + [(r, draft[r])]
    start, slots = _place(rng, runs)
    seg_starts, seg_lens = [[] for _ in range(b)], [[] for _ in range(b)]
    for (r, x), at in zip(runs, start):
        seg_starts[r].append(int(at))
        seg_lens[r].append(int(x))
    t_max, k_max = max(draft), max(p + t for p, t in zip(prior, draft))
    key_slots = np.zeros((b, k_max), dtype=np.int64)
    vis = np.zeros((b, t_max, t_max), dtype=bool)
    rows = np.zeros((b, t_max), dtype=np.int64)
    trees, at = [], 0
    for r in range(b):
        slot = np.concatenate([a + np.arange(x) for a, x in zip(seg_starts[r], seg_lens[r])])
        key_slots[r, :len(slot)] = slot
        key_slots[r, len(slot):] = slot[0]
        t = draft[r]
        if case["form"] == "mask":
            m = np.tril(rng.rand(t, t) < 0.5)
            m[np.arange(t), np.arange(t)] = True
            trees.append(m)
            vis[r, :t, :t] = m
        else:
            trees.append(_parents(rng, t, case["form"]))
            vis[r, :t, :t] = _ancestors(trees[-1])
        rows[r, :t] = at + np.arange(t)
        at += t
    to = lambda x: torch.from_numpy(x).to(DEV)
    s.update(draft=draft, prior=prior, trees=trees, seg_starts=seg_starts, seg_lens=seg_lens)
    s["key_slots"], s["visible"], s["rows"] = to(key_slots), to(vis), to(rows)
    s["packed"] = to(np.concatenate([r * t_max + np.arange(t) for r, t in enumerate(draft)]))
    s["prior_dev"], s["draft_dev"] = to(np.array(prior)), to(np.array(draft))
    s["q"] = _normal(gen, at, hq, d)
    s["k_pool"] = _pool(gen, slots, hk, d, case["fp8"])
    s["v_pool"] = _pool(gen, slots, hk, d, case["fp8"])
    s["k_scale"], s["v_scale"], s["scale"] = _scales(hk), _scales(hk) * 1.5, 1 / math.sqrt(d)
    if own:
        import segmented_kv_cache_b200 as sa
        kw = ({"mask": np.concatenate([m.reshape(-1) for m in trees])} if case["form"] == "mask"
              else {"parents": [p for t in trees for p in t]})
        tab = sa.TreeTable.build(draft, seg_starts, seg_lens, slots, hq, hk, d, **kw).to(DEV)
        s["table"] = tab
        s["workspace"] = torch.empty(max(16, tab.workspace_bytes), dtype=torch.uint8, device=DEV)
        s["out"] = torch.empty_like(s["q"])
        s["lse"] = torch.empty(at, hq, dtype=torch.float32, device=DEV)


# ------------------------------------------------------------------------------- plain form
def _rotate(x, s, backward=False):
    """Rotary positions of x [n, heads, d]: angles in 64 bits, products in 32."""
    c = s["case"]
    r, half = c["rotary"], c["rotary"] // 2
    angle = s["positions"].double()[:, None] * s["inv_freq"]
    cos = (torch.cos(angle) * s["amp"]).float()[:, None]
    sin = (torch.sin(angle) * s["amp"]).float()[:, None]
    sin = -sin if backward else sin
    x = x.float()
    if c["interleaved"]:
        a, b = x[..., 0:r:2], x[..., 1:r:2]
        turned = torch.stack([a * cos - b * sin, b * cos + a * sin], dim=-1).flatten(-2)
    else:
        a, b = x[..., :half], x[..., half:r]
        turned = torch.cat([a * cos - b * sin, b * cos + a * sin], dim=-1)
    return torch.cat([turned, x[..., r:]], dim=-1)


def _e4m3(x, scale):
    return (x / scale[:, None]).clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)


def _values(pool, fp8):
    """What the caller sees of a pool: E4M3 codes as the numbers they stand for."""
    return pool.view(torch.float8_e4m3fn) if fp8 else pool


def _plain_tree(s):
    c = s["case"]
    hq, hk, d = c["q_heads"], c["kv_heads"], c["head_dim"]
    b, t = s["rows"].shape
    k, v = s["k_pool"], s["v_pool"]
    if c["fp8"]:
        k, v = k.view(torch.float8_e4m3fn), v.view(torch.float8_e4m3fn)
    gather = lambda pool: pool.view(torch.uint8 if c["fp8"] else pool.dtype)[s["key_slots"]]
    kk, vv = gather(k), gather(v)
    if c["fp8"]:
        kk = kk.view(torch.float8_e4m3fn).float() * s["k_scale"][:, None]
        vv = vv.view(torch.float8_e4m3fn).float() * s["v_scale"][:, None]
    kk, vv = kk.float().transpose(1, 2), vv.float().transpose(1, 2)   # [b, hk, keys, d]
    q = s["q"][s["rows"]].float().view(b, t, hk, hq // hk, d).permute(0, 2, 3, 1, 4)
    n = kk.shape[2]
    score = torch.matmul(q.reshape(b, hk, -1, d), kk.transpose(2, 3)) * s["scale"]
    score = score.view(b, hk, hq // hk, t, n)
    at = torch.arange(n, device=DEV)[None] - s["prior_dev"][:, None]   # place among the drafts
    seen = torch.gather(s["visible"], 2, at.clamp(0, t - 1)[:, None].expand(b, t, n))
    seen = (seen & (at >= 0)[:, None] & (at < s["draft_dev"][:, None])[:, None]) | (at < 0)[:, None]
    score = score.masked_fill(~seen[:, None, None], float("-inf"))
    top = score.amax(-1, keepdim=True)
    top = top.masked_fill(top == float("-inf"), 0.0)
    p = torch.exp(score - top)
    total = p.sum(-1, keepdim=True)
    o = torch.matmul(p.view(b, hk, -1, n), vv).view(b, hk, hq // hk, t, d) / total.clamp(min=1e-30)
    lse = (top + torch.log(total))[..., 0]
    o = o.permute(0, 3, 1, 2, 4).reshape(b * t, hq, d)[s["packed"]]
    lse = lse.permute(0, 3, 1, 2).reshape(b * t, hq)[s["packed"]]
    return {"out": o.to(torch.bfloat16), "lse": lse}


def run(s):
    if own:
        return _run_own(s)
    c = s["case"]
    if c["op"] == "rope":
        return _rotate(s["x"], s, c["backward"]).to(torch.bfloat16)
    if c["op"] == "append":
        q, k, v = _rotate(s["q"], s).to(torch.bfloat16), _rotate(s["k"], s), s["v"]
        if c["fp8"]:
            k, v = _e4m3(k, s["k_scale"]), _e4m3(v.float(), s["v_scale"])
        s["k_pool"][s["slots"].long()] = k.to(s["k_pool"].dtype)
        s["v_pool"][s["slots"].long()] = v
        return {"q": q, "k_pool": _values(s["k_pool"], c["fp8"]),
                "v_pool": _values(s["v_pool"], c["fp8"])}
    if c["op"] == "move":
        src, dst = s["src"].long(), s["dst"].long()
        s["k_pool"][dst] = s["k_pool"][src]
        s["v_pool"][dst] = s["v_pool"][src]
        return {"k_pool": _values(s["k_pool"], c["fp8"]), "v_pool": _values(s["v_pool"], c["fp8"])}
    return _plain_tree(s)


# ------------------------------------------------------------------------------- the library
def _run_own(s):
    import segmented_kv_cache_b200 as sa
    c = s["case"]
    if c["op"] == "rope":
        sa.seg_attn_rope(s["x"], s["out"], s["positions"], s["rope"], backward=c["backward"])
        return s["out"]
    if c["op"] == "append":
        if c["fp8"]:
            sa.seg_attn_rope_append_fp8(s["q"], s["q_out"], s["k"], s["v"], s["positions"],
                                        s["slots"], s["rope"], s["k_scale"], s["v_scale"],
                                        s["k_pool"], s["v_pool"])
        else:
            sa.seg_attn_rope_append(s["q"], s["q_out"], s["k"], s["v"], s["positions"],
                                    s["slots"], s["rope"], s["k_pool"], s["v_pool"])
        return {"q": s["q_out"], "k_pool": _values(s["k_pool"], c["fp8"]),
                "v_pool": _values(s["v_pool"], c["fp8"])}
    if c["op"] == "move":
        sa.seg_attn_kv_move(s["k_pool"], s["v_pool"], s["src"], s["dst"], s["offsets"])
        return {"k_pool": _values(s["k_pool"], c["fp8"]), "v_pool": _values(s["v_pool"], c["fp8"])}
    tab = s["table"]
    if c["fp8"]:
        sa.seg_attn_tree_fp8(s["q"], s["k_pool"], s["v_pool"], s["k_scale"], s["v_scale"],
                             s["out"], s["lse"], tab.device, tab.desc, s["scale"], s["workspace"])
    else:
        sa.seg_attn_tree(s["q"], s["k_pool"], s["v_pool"], s["out"], s["lse"], tab.device,
                         tab.desc, s["scale"], s["workspace"])
    return {"out": s["out"], "lse": s["lse"]}


# ------------------------------------------------------------------------------- 64 bits
def _exact_angles(case, positions):
    """Angle of every (token, pair), from the definition of each scaling; and the amplitude."""
    r, base, f = case["rotary"], case["base"], case["factor"]
    theta, amp = [], 1.0
    if case["scaling"] == "yarn":
        amp = 1.0 + math.log(f) / 10
    for i in range(r // 2):
        w = base ** (-2 * i / r)
        if case["scaling"] == "ntk" and r > 2:
            w = (base * f ** (r / (r - 2))) ** (-2 * i / r)
        elif case["scaling"] == "linear":
            w = w / f
        elif case["scaling"] == "yarn":
            edge = [r / 2 * math.log(ORIGINAL / (2 * math.pi * n)) / math.log(base)
                    for n in (YARN_HIGH, YARN_LOW)]
            lo, hi = max(math.floor(edge[0]), 0), min(math.ceil(edge[1]), r - 1)
            mix = min(max((i - lo) / max(hi - lo, 1e-3), 0.0), 1.0)
            w = w * (1 - mix) + w / f * mix
        elif case["scaling"] == "wavelength":
            wavelength = 2 * math.pi / w
            if wavelength > ORIGINAL / WAVE_LOW:
                w = w / f
            elif wavelength >= ORIGINAL / WAVE_HIGH:
                mix = (ORIGINAL / wavelength - WAVE_LOW) / (WAVE_HIGH - WAVE_LOW)
                w = (1 - mix) * w / f + mix * w
        theta.append(w)
    return positions.double()[:, None] * torch.tensor(theta, dtype=torch.float64, device=DEV), amp


def _exact_rotate(x, s, sign=1.0):
    """Each pair as a complex number, turned by its angle."""
    c = s["case"]
    angle, amp = _exact_angles(c, s["positions"])
    x = x.double().clone()
    r = c["rotary"]
    first = torch.arange(0, r, 2) if c["interleaved"] else torch.arange(r // 2)
    second = first + (1 if c["interleaved"] else r // 2)
    z = torch.complex(x[..., first], x[..., second])
    z = z * torch.polar(torch.full_like(angle, amp), sign * angle)[:, None]
    x[..., first], x[..., second] = z.real, z.imag
    return x


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "rope":
        return _exact_rotate(s["x"], s, -1.0 if case["backward"] else 1.0)
    if case["op"] in ("append", "move"):
        see = lambda p: (p.view(torch.float8_e4m3fn) if case["fp8"] else p).double()
        k_pool, v_pool = see(s["k_pool"]), see(s["v_pool"])
        if case["op"] == "move":
            dst, src = s["dst"].long(), s["src"].long()
            k_pool[dst], v_pool[dst] = k_pool[src], v_pool[src]
            return {"k_pool": k_pool, "v_pool": v_pool}
        k, v, at = _exact_rotate(s["k"], s), s["v"].double(), s["slots"].long()
        if case["fp8"]:   # in the cache's units, before the rounding to a code
            k, v = k / s["k_scale"].double()[:, None], v / s["v_scale"].double()[:, None]
            k, v = k.clamp(-448, 448), v.clamp(-448, 448)
        k_pool[at], v_pool[at] = k, v
        return {"q": _exact_rotate(s["q"], s), "k_pool": k_pool, "v_pool": v_pool}
    return _exact_tree(s)


def _exact_tree(s):
    c = s["case"]
    hq, hk = c["q_heads"], c["kv_heads"]
    outs, lses, at = [], [], 0
    for r, t in enumerate(s["draft"]):
        n = s["prior"][r] + t
        slot = torch.cat([torch.arange(a, a + x) for a, x in
                          zip(s["seg_starts"][r], s["seg_lens"][r])]).to(DEV)
        k, v = s["k_pool"][slot], s["v_pool"][slot]
        if c["fp8"]:
            k = k.view(torch.float8_e4m3fn).double() * s["k_scale"].double()[:, None]
            v = v.view(torch.float8_e4m3fn).double() * s["v_scale"].double()[:, None]
        k, v = k.double(), v.double()
        seen = np.ones((t, n), dtype=bool)
        tree = s["trees"][r]
        if c["form"] == "mask":
            seen[:, n - t:] = tree
        else:
            seen[:, n - t:] = False
            for i in range(t):
                j = i
                while j >= 0:
                    seen[i, n - t + j] = True
                    j = tree[j]
        hide = ~torch.from_numpy(seen).to(DEV)
        q = s["q"][at:at + t].double()
        at += t
        o = torch.empty_like(q)
        lse = torch.empty(t, hq, dtype=torch.float64, device=DEV)
        for g in range(hk):
            heads = slice(g * (hq // hk), (g + 1) * (hq // hk))
            x = torch.einsum("thd,kd->thk", q[:, heads], k[:, g]) / math.sqrt(c["head_dim"])
            x = x.masked_fill(hide[:, None], float("-inf"))
            lse[:, heads] = torch.logsumexp(x, -1)
            o[:, heads] = torch.einsum("thk,kd->thd", torch.softmax(x, -1), v[:, g])
        outs.append(o)
        lses.append(lse)
    return {"out": torch.cat(outs), "lse": torch.cat(lses)}
