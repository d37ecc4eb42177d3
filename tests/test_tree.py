"""Attention of drafted tokens, row moves, and a whole drafting step on the GPU, against 64 bits."""
import math
import random

import pytest
import torch

import segmented_kv_cache_b200 as sa

import draft_reference as ref

pytestmark = pytest.mark.gpu


def run(c, tab, lse=True, stream=None, ws=None):
    out = torch.full_like(c["q"], math.nan)
    ls = torch.full(c["q"].shape[:2], math.nan, dtype=torch.float32, device="cuda") if lse else None
    if ws is None:
        ws = torch.full((max(16, tab.workspace_bytes),), 0xFF, dtype=torch.uint8, device="cuda")
    if c["fp8"]:
        sa.seg_attn_tree_fp8(c["q"], c["k_pool"], c["v_pool"], c["k_scale"], c["v_scale"], out, ls,
                             tab.device, tab.desc, c["scale"], ws, stream)
    else:
        sa.seg_attn_tree(c["q"], c["k_pool"], c["v_pool"], out, ls, tab.device, tab.desc, c["scale"],
                         ws, stream)
    return out, ls


def table(c, **kw):
    hq, d = c["q"].shape[1:]
    return sa.TreeTable.build(c["draft"], c["seg_starts"], c["seg_lens"], c["num_slots"], hq,
                              c["k_pool"].shape[1], d, **kw).to("cuda")


def check(c, what="", **kw):
    out, lse = run(c, table(c, **kw))
    want = ref.tree(c["q"], c["k_values"], c["v_values"], c["draft"], ref.visible(c["draft"], **kw),
                    c["seg_starts"], c["seg_lens"], c["scale"])
    ref.check_tree(out, lse, want, what)
    assert sa.seg_attn_take_device_error() == 0
    return out, lse


HEADS = [(64, 8, 128), (8, 1, 64), (4, 4, 128), (16, 2, 64), (128, 1, 64), (6, 3, 128), (32, 1, 128)]


@pytest.mark.parametrize("hq,hkv,d", HEADS)
@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("form", ["parents", "mask", "chain"])
def test_mixed_batch(hq, hkv, d, fp8, form):
    rnd = random.Random(f"{hq}{hkv}{d}{fp8}{form}")
    draft = [1, 7, 0, 32, 33, 3, 65]
    prior = [1000, 0, 50, 127, 128, 129, 700]
    c = ref.tree_case(rnd, draft, prior, hq, hkv, d, fp8=fp8)
    kw = {}
    if form == "parents":
        kw = dict(parents=[p for t in draft for p in ref.random_parents(rnd, t)])
    elif form == "mask":
        kw = dict(mask=[rnd.random() < 0.4 for _ in range(sum(t * t for t in draft))])
    check(c, f"{hq}/{hkv} d{d} fp8={fp8} {form}", **kw)


@pytest.mark.parametrize("prior", [0, 1, 5, 127, 128, 129, 1024, 5000, 20001])
@pytest.mark.parametrize("fp8", [False, True])
def test_single_token(prior, fp8):
    c = ref.tree_case(random.Random(prior), [1], [prior], 64, 8, 128, nseg=5, fp8=fp8)
    check(c, f"one token over {prior}")


def test_single_tokens_match_decode():
    """A draft of one token is a decode: same values to the two kernels' rounding."""
    c = ref.tree_case(random.Random(1), [1] * 5, [300, 1, 2000, 64, 4095], 16, 2, 128)
    out, lse = check(c)
    tab = sa.SegTable.build(None, c["seg_starts"], c["seg_lens"], c["num_slots"], True,
                            sa.MODE_DECODE, 16, 2, 128).to("cuda")
    o2, l2 = torch.empty_like(out), torch.empty_like(lse)
    ws = torch.empty(max(16, tab.workspace_bytes), dtype=torch.uint8, device="cuda")
    sa.seg_attn_decode(c["q"], c["k_pool"], c["v_pool"], o2, l2, tab.device, tab.desc, c["scale"], ws)
    assert float((lse - l2).abs().max()) <= 6e-4
    assert float((out.float() - o2.float()).abs().max()) <= 2e-2


def test_chain_matches_causal_prefill():
    c = ref.tree_case(random.Random(2), [40, 9], [777, 3000], 16, 2, 128)
    out, lse = check(c)
    tab = sa.SegTable.build(c["draft"], c["seg_starts"], c["seg_lens"], c["num_slots"], True,
                            sa.MODE_PREFILL, 16, 2, 128).to("cuda")
    o2, l2 = torch.empty_like(out), torch.empty_like(lse)
    ws = torch.empty(max(16, tab.workspace_bytes), dtype=torch.uint8, device="cuda")
    sa.seg_attn_prefill(c["q"], c["k_pool"], c["v_pool"], o2, l2, tab.device, tab.desc, c["scale"], ws)
    assert float((lse - l2).abs().max()) <= 6e-4
    assert float((out.float() - o2.float()).abs().max()) <= 2e-2


@pytest.mark.parametrize("draft,hq,hkv,d", [([300], 64, 8, 128), ([257, 1], 128, 1, 64),
                                            ([1024], 2, 1, 64)])
def test_large_trees(draft, hq, hkv, d):
    rnd = random.Random(sum(draft))
    c = ref.tree_case(rnd, draft, [600] * len(draft), hq, hkv, d)
    check(c, parents=[p for t in draft for p in ref.random_parents(rnd, t)])


def test_long_context_in_many_pieces_and_segments():
    c = ref.tree_case(random.Random(5), [12], [70000], 8, 1, 128, nseg=40)
    tab = table(c)
    assert tab.desc.pass_.num_work > 30
    check(c, parents=[-1, 0, 0, 1, 1, 2, 3, 3, 4, 5, 6, 6])


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("draft", [4, 40])
def test_a_copy_that_never_lands_is_an_error_not_a_hang(fp8, draft):
    """The stall test withholds K tile 2: every CTA gives up after 1 ms (one query tile, whose two
    softmax groups meet at the end, and two), the error word says so, and the next call is right."""
    c = ref.tree_case(random.Random(15), [draft] * 20, [1500] * 20, 64, 8, 128, fp8=fp8)
    tab = table(c)
    assert tab.desc.pass_.max_k_tiles > 2
    sa.seg_attn_stall_test(2, 1000)
    try:
        run(c, tab)
        torch.cuda.synchronize()
        assert sa.seg_attn_take_device_error() == 1
    finally:
        sa.seg_attn_stall_test(-1, 1000000)
    check(c)


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("short", [1, 3, 40])
def test_many_short_segments(fp8, short):
    """More segments than a producer warp holds at once, inside one K tile and across tiles; empty
    segments among them."""
    rnd = random.Random(short)
    draft, prior = [5, 17], [700, 1500]
    c = ref.tree_case(rnd, draft, prior, 16, 2, 128, fp8=fp8)
    starts, lens = [], []
    for ss, ll in zip(c["seg_starts"], c["seg_lens"]):
        s2, l2 = [], []
        for s, l in zip(ss, ll):   # the same slots, cut into runs of up to `short` keys
            at = 0
            while at < l:
                n = min(l - at, rnd.randint(1, short))
                if rnd.random() < 0.2:
                    s2.append(rnd.randrange(c["num_slots"]))
                    l2.append(0)
                s2.append(s + at)
                l2.append(n)
                at += n
        starts.append(s2)
        lens.append(l2)
    # runs in another order: neighbouring keys no longer sit in neighbouring slots
    for r in range(2):
        order = list(range(len(starts[r])))
        rnd.shuffle(order)
        starts[r], lens[r] = [starts[r][i] for i in order], [lens[r][i] for i in order]
    c["seg_starts"], c["seg_lens"] = starts, lens
    assert len(starts[1]) > 32 or short == 40
    check(c, f"runs of {short}", parents=[p for t in draft for p in ref.random_parents(rnd, t)])
    # the plain prefill walks the same segments
    hq, d = c["q"].shape[1:]
    tab = sa.SegTable.build(draft, starts, lens, c["num_slots"], True, sa.MODE_PREFILL, hq, 2, d).to("cuda")
    out, lse = torch.empty_like(c["q"]), torch.empty(22, hq, device="cuda")
    ws = torch.empty(max(16, tab.workspace_bytes), dtype=torch.uint8, device="cuda")
    if fp8:
        sa.seg_attn_prefill_fp8(c["q"], c["k_pool"], c["v_pool"], c["k_scale"], c["v_scale"], out, lse,
                                tab.device, tab.desc, c["scale"], ws)
    else:
        sa.seg_attn_prefill(c["q"], c["k_pool"], c["v_pool"], out, lse, tab.device, tab.desc, c["scale"], ws)
    want = ref.tree(c["q"], c["k_values"], c["v_values"], draft, ref.visible(draft), starts, lens, c["scale"])
    ref.check_tree(out, lse, want, "prefill")


@pytest.mark.parametrize("fp8", [False, True])
def test_rows_that_see_nothing(fp8):
    """An empty mask row sees the cached keys only, or, without any, nothing: 0 and -inf."""
    draft, prior = [4, 3], [0, 200]
    m = [[1, 0, 0, 0], [0, 0, 0, 0], [1, 1, 0, 1], [0, 0, 0, 0]]
    mask = [x for row in m for x in row] + [0] * 9
    c = ref.tree_case(random.Random(6), draft, prior, 16, 2, 64, fp8=fp8)
    out, lse = check(c, mask=mask)
    for i in (1, 3):
        assert torch.equal(out[i], torch.zeros_like(out[i])) and bool((lse[i] == -math.inf).all())
    assert bool(torch.isfinite(lse[4:]).all())


@pytest.mark.parametrize("value", [math.nan, math.inf, -math.inf, torch.finfo(torch.bfloat16).min])
def test_masked_rows_may_hold_anything(value):
    """What a token does not see never reaches its row; V's NaN and infinities reach those that
    see them."""
    rnd = random.Random(7)
    draft, prior = [6, 5, 50, 150], [130, 0, 4000, 60]
    parents = [-1, 0, 0, 1, 2, 4, -1, -1, 1, 2, 2] + [p for t in draft[2:] for p in
                                                      ref.random_parents(rnd, t)]
    c = ref.tree_case(rnd, draft, prior, 16, 2, 128)
    clean, clean_lse = check(c, parents=parents)
    vis = ref.visible(draft, parents=parents)
    for r, j in ((0, 1), (0, 5), (1, 0), (1, 2), (2, 0), (2, 33), (3, 10), (3, 67), (3, 149)):
        keys = [s + i for s, l in zip(c["seg_starts"][r], c["seg_lens"][r]) for i in range(l)]
        slot = keys[prior[r] + j]
        for name in ("k_pool", "v_pool"):
            keep = c[name][slot].clone()
            c[name][slot] = value
            out, lse = run(c, table(c, parents=parents))
            c[name][slot] = keep
            at = sum(draft[:r])
            sees = torch.zeros(sum(draft), dtype=torch.bool)
            sees[at:at + draft[r]] = torch.from_numpy(vis[r][:, j])
            sees = sees.cuda()
            assert torch.equal(out[~sees], clean[~sees]) and torch.equal(lse[~sees], clean_lse[~sees])
            if math.isinf(value) and name == "v_pool":
                assert bool((out[sees] == value).all())
            if math.isnan(value):
                assert bool(torch.isnan(out[sees]).all())
                assert torch.isnan(lse[sees]).all() if name == "k_pool" else \
                    torch.equal(lse[sees], clean_lse[sees])


def test_lse_is_optional_and_repeats_are_bit_equal():
    c = ref.tree_case(random.Random(8), [9, 20], [3000, 500], 64, 8, 128)
    tab = table(c)
    a, la = run(c, tab)
    b, lb = run(c, tab)
    d, none = run(c, tab, lse=False)
    assert none is None and torch.equal(a, b) and torch.equal(a, d) and torch.equal(la, lb)


def test_two_streams_with_workspaces_of_their_own():
    c1 = ref.tree_case(random.Random(9), [16] * 4, [3000] * 4, 64, 8, 128)
    c2 = ref.tree_case(random.Random(10), [5] * 6, [2000] * 6, 64, 8, 128, fp8=True)
    want = [run(c, table(c)) for c in (c1, c2)]
    tabs = [table(c1), table(c2)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    got = [[], []]
    outs = []
    for c, tab, s in zip((c1, c2), tabs, streams):
        with torch.cuda.stream(s):
            ws = torch.empty(max(16, tab.workspace_bytes), dtype=torch.uint8, device="cuda")
            outs.append([run(c, tab, ws=ws) for _ in range(6)])
    torch.cuda.synchronize()
    for runs, (o, l) in zip(outs, want):
        for a, b in runs:
            assert torch.equal(a, o) and torch.equal(b, l)


def test_captured_and_replayed_with_new_values():
    c = ref.tree_case(random.Random(11), [7, 12], [900, 260], 16, 2, 128)
    parents = [-1, 0, 0, 1, 1, 2, 3] + [i - 1 for i in range(12)]
    tab = table(c, parents=parents)
    ws = torch.empty(max(16, tab.workspace_bytes), dtype=torch.uint8, device="cuda")
    out, lse = torch.empty_like(c["q"]), torch.empty(19, 16, device="cuda")
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        sa.seg_attn_tree(c["q"], c["k_pool"], c["v_pool"], out, lse, tab.device, tab.desc, c["scale"], ws)
    for k in range(3):
        c["q"].normal_()
        c["v_pool"].mul_(1.25)
        graph.replay()
        torch.cuda.synchronize()
        want = ref.tree(c["q"], c["k_values"], c["v_values"], c["draft"],
                        ref.visible(c["draft"], parents=parents), c["seg_starts"], c["seg_lens"],
                        c["scale"])
        ref.check_tree(out, lse, want, f"replay {k}")


def test_binding_refuses_wrong_tensors():
    c = ref.tree_case(random.Random(12), [3], [3000], 4, 2, 64)
    tab = table(c)
    out, lse = torch.empty_like(c["q"]), torch.empty(3, 4, device="cuda")
    assert tab.workspace_bytes > 0
    ws = torch.empty(max(16, tab.workspace_bytes), dtype=torch.uint8, device="cuda")
    good = dict(q=c["q"], k_pool=c["k_pool"], v_pool=c["v_pool"], out=out, lse=lse,
                dev_table=tab.device, desc=tab.desc, softmax_scale=0.1, workspace=ws)
    sa.seg_attn_tree(**good)
    bad = [dict(q=c["q"].float()), dict(q=c["q"][:2]), dict(out=out.cpu()), dict(lse=lse.double()),
           dict(lse=lse[:2]), dict(k_pool=c["k_pool"][1:]), dict(v_pool=c["v_pool"].view(torch.uint8)),
           dict(dev_table=tab.device[:8]), dict(dev_table=tab.host),
           dict(q=c["q"].transpose(0, 1).contiguous().transpose(0, 1))]
    for kw in bad:
        with pytest.raises(sa.SegAttnError) as e:
            sa.seg_attn_tree(**{**good, **kw})
        assert e.value.code == sa.STATUS["INVALID_ARG"], list(kw)
    with pytest.raises(sa.SegAttnError) as e:
        sa.seg_attn_tree(**{**good, "workspace": None})
    assert e.value.code == sa.STATUS["WORKSPACE"]


# ----------------------------------------------------------------------------- row moves
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.uint8])
@pytest.mark.parametrize("hk,d", [(8, 128), (1, 64), (3, 48), (32, 128)])
@pytest.mark.parametrize("grouped", [False, True])
def test_move_disjoint_rows(dtype, hk, d, grouped):
    g = torch.Generator().manual_seed(hk + d)
    S, n = 500, 180
    pools = [torch.randint(0, 256, (S, hk, d * (2 if dtype is torch.bfloat16 else 1)), generator=g,
                           dtype=torch.uint8) for _ in range(2)]
    perm = torch.randperm(S, generator=g)
    src, dst = perm[:n].to(torch.int32), perm[n:2 * n].to(torch.int32)
    want = [p.clone() for p in pools]
    for w, p in zip(want, pools):
        w[dst.long()] = p[src.long()]
    dev = [p.cuda().view(dtype) for p in pools]
    offsets = torch.tensor([0, 0, 1, 9, 10, 60, 60, 180], dtype=torch.int32).cuda() if grouped else None
    sa.seg_attn_kv_move(dev[0], dev[1], src.cuda(), dst.cuda(), offsets)
    for w, p in zip(want, dev):
        assert torch.equal(p.view(torch.uint8).cpu(), w)
    assert sa.seg_attn_take_device_error() == 0


def test_move_accepted_rows_to_the_front_in_place():
    """Sources later in the list than destinations, overlapping: rows move down in order."""
    g = torch.Generator().manual_seed(3)
    S, hk, d, B, T = 400, 2, 64, 5, 40
    k, v = (torch.randn(S, hk, d, generator=g).to(torch.bfloat16) for _ in range(2))
    src, dst, off = [], [], [0]
    wk, wv = k.clone(), v.clone()
    for r in range(B):
        path = sorted(torch.randperm(T, generator=g)[: (1, 8, 9, 17, 40)[r]].tolist())
        src += [r * T + p for p in path]
        dst += [r * T + i for i in range(len(path))]
        off.append(len(src))
    for a, b in zip(src, dst):
        wk[b], wv[b] = wk[a].clone(), wv[a].clone()
    kd, vd = k.cuda(), v.cuda()
    i32 = lambda x: torch.tensor(x, dtype=torch.int32).cuda()
    sa.seg_attn_kv_move(kd, vd, i32(src), i32(dst), i32(off))
    assert torch.equal(kd.cpu(), wk) and torch.equal(vd.cpu(), wv)


def test_move_skips_padding_and_flags_slots_out_of_range():
    S, hk, d = 20, 2, 64
    k = torch.arange(S, device="cuda", dtype=torch.float32)[:, None, None].expand(S, hk, d).to(
        torch.bfloat16).contiguous()
    v = k + 100
    i32 = lambda x: torch.tensor(x, dtype=torch.int32).cuda()
    pad_src, pad_dst = i32([-1, 4, 2, 7]), i32([-1, 9, 2, 11])
    sa.seg_attn_kv_move(k, v, pad_src, pad_dst)
    assert sa.seg_attn_take_device_error() == 0
    assert k[:, 0, 0].tolist() == [0, 1, 2, 3, 4, 5, 6, 7, 8, 4, 10, 7] + list(range(12, 20))
    before = k.clone()
    sa.seg_attn_kv_move(k, v, i32([S, 3, -2, 5]), i32([3, S, 1, -7]))
    assert sa.seg_attn_take_device_error() == 2 and sa.seg_attn_take_device_error() == 0
    assert torch.equal(k, before)
    # offsets past the list are clamped; an empty list does nothing
    sa.seg_attn_kv_move(k, v, i32([0]), i32([15]), i32([-5, 1, 99]))
    assert float(k[15, 0, 0]) == 0.0
    sa.seg_attn_kv_move(k, v, i32([]), i32([]))
    with pytest.raises(sa.SegAttnError):
        sa.seg_attn_kv_move(k, v, i32([1]), i32([1, 2]))
    with pytest.raises(sa.SegAttnError):
        sa.seg_attn_kv_move(k.float(), v.float(), i32([1]), i32([2]))


# ----------------------------------------------------------------------------- a drafting step
@pytest.mark.parametrize("fp8", [False, True])
def test_draft_verify_commit_steps(fp8):
    """Three steps of drafting over an allocator-managed cache: append the rotated drafts to
    scratch slots, attend as a tree, move an accepted path to each request's own run.  The
    attention of every step is checked against 64 bits on the cache as it should be, kept
    apart as plain lists of (key, value) rows."""
    rnd = random.Random(20)
    g = torch.Generator().manual_seed(20)
    hq, hk, d, S, B, T = 16, 2, 128, 3000, 3, 10
    dtype = torch.uint8 if fp8 else torch.bfloat16
    kp, vp = (torch.zeros(S, hk, d, dtype=dtype, device="cuda") for _ in range(2))
    ks, vs = torch.tensor([0.06, 0.08]).cuda(), torch.tensor([0.05, 0.07]).cuda()
    plan = sa.seg_attn_rope_plan(d)
    pool = sa.SegPool(S)
    scratch = {r: torch.from_numpy(pool.append(1000 + r, T)).cuda() for r in range(B)}
    lens, truth = [0] * B, [[] for _ in range(B)]   # truth: (k, v) rows as stored

    def append(q, k, v, pos, slots):
        q_out = torch.empty_like(q) if q is not None else None
        if fp8:
            sa.seg_attn_rope_append_fp8(q, q_out, k, v, pos, slots, plan, ks, vs, kp, vp)
        else:
            sa.seg_attn_rope_append(q, q_out, k, v, pos, slots, plan, kp, vp)
        return q_out

    values = lambda p, s: (p.view(torch.float8_e4m3fn).double() * s.double()[:, None]) if fp8 else p.double()

    def stored(slots):
        i = slots.long()
        return list(zip(values(kp, ks)[i], values(vp, vs)[i]))

    for r, n in enumerate((300, 1, 515)):   # prompts
        slots = torch.from_numpy(pool.append(r, n)).cuda()
        x = torch.randn(n, 2 * hk, d, generator=g).to(torch.bfloat16).cuda()
        append(None, x[:, :hk], x[:, hk:], torch.arange(n, dtype=torch.int32).cuda(), slots)
        truth[r] += stored(slots)
        lens[r] = n
    for step in range(3):
        parents = [ref.random_parents(rnd, T) for _ in range(B)]
        depth = []
        for p in parents:
            dd = []
            for x in p:
                dd.append(0 if x < 0 else dd[x] + 1)
            depth.append(dd)
        pos = torch.tensor([lens[r] + depth[r][i] for r in range(B) for i in range(T)],
                           dtype=torch.int32).cuda()
        slots = torch.cat([scratch[r] for r in range(B)])
        qkv = torch.randn(B * T, hq + 2 * hk, d, generator=g).to(torch.bfloat16).cuda()
        q = append(qkv[:, :hq], qkv[:, hq:hq + hk], qkv[:, hq + hk:], pos, slots)
        y, mag = ref.rope(qkv[:, :hq], pos, ref.plain_freq(d))
        assert bool(((q.double().cpu() - y).abs() <= ref.rope_tolerance(y, mag) + 1e-30).all())
        segs = [pool.segments(r) for r in range(B)]
        own = [pool.segments(1000 + r) for r in range(B)]
        starts = [a[0] + b[0] for a, b in zip(segs, own)]
        ll = [a[1] + b[1] for a, b in zip(segs, own)]
        tab = sa.TreeTable.build([T] * B, starts, ll, S, hq, hk, d,
                                 parents=[x for p in parents for x in p]).to("cuda")
        c = dict(q=q, k_pool=kp, v_pool=vp, k_scale=ks, v_scale=vs, scale=1 / math.sqrt(d), fp8=fp8)
        out, lse = run(c, tab)
        # the cache as it should be: every request's rows in order, then its drafts
        rows, k_starts, k_lens = [], [], []
        for r in range(B):
            k_starts.append([len(rows)])
            rows += truth[r] + stored(scratch[r])
            k_lens.append([len(rows) - k_starts[-1][0]])
        want = ref.tree(q, torch.stack([k for k, _ in rows]), torch.stack([v for _, v in rows]),
                        [T] * B, ref.visible([T] * B, parents=[x for p in parents for x in p]),
                        k_starts, k_lens, c["scale"])
        ref.check_tree(out, lse, want, f"step {step}")
        # accept a random path from a root to some token
        src, dst, off = [], [], [0]
        for r in range(B):
            path, x = [], rnd.randrange(T)
            while x >= 0:
                path.append(x)
                x = parents[r][x]
            path.reverse()
            new = pool.append(r, len(path))
            src += [int(scratch[r][i]) for i in path]
            dst += new.tolist()
            off.append(len(src))
            truth[r] += [stored(scratch[r][i:i + 1])[0] for i in path]
            lens[r] += len(path)
        i32 = lambda v: torch.tensor(v, dtype=torch.int32).cuda()
        sa.seg_attn_kv_move(kp, vp, i32(src), i32(dst), i32(off))
    for r in range(B):
        s, l = pool.segments(r)
        slots = torch.tensor([a + i for a, n in zip(s, l) for i in range(n)]).cuda()
        got = stored(slots)
        assert len(got) == len(truth[r]) == lens[r]
        assert all(torch.equal(a, x) and torch.equal(b, y) for (a, b), (x, y) in zip(got, truth[r]))
    assert sa.seg_attn_take_device_error() == 0


def test_masked_nan_codes_in_an_e4m3_cache():
    """E4M3 has NaN codes only: a drafted V row with some reaches the rows that see it, in those
    columns, and no others; a K row with some never reaches rows that do not see it."""
    rnd = random.Random(13)
    draft, prior = [9, 40], [300, 0]
    parents = [p for t in draft for p in ref.random_parents(rnd, t)]
    c = ref.tree_case(rnd, draft, prior, 64, 8, 128, fp8=True)
    clean, clean_lse = check(c, parents=parents)
    vis = ref.visible(draft, parents=parents)
    for r, j in ((0, 0), (0, 7), (1, 3), (1, 39)):
        keys = [s + i for s, l in zip(c["seg_starts"][r], c["seg_lens"][r]) for i in range(l)]
        slot = keys[prior[r] + j]
        at = sum(draft[:r])
        sees = torch.zeros(sum(draft), dtype=torch.bool)
        sees[at:at + draft[r]] = torch.from_numpy(vis[r][:, j])
        sees = sees.cuda()
        for name, code in (("v_pool", 0x7F), ("v_pool", 0xFF), ("k_pool", 0x7F)):
            keep = c[name][slot].clone()
            c[name][slot, 2, 5] = code
            out, lse = run(c, table(c, parents=parents))
            c[name][slot] = keep
            same = (out == clean)
            hit = torch.zeros_like(same)
            if name == "v_pool":
                hit[sees, 16:24, 5] = True          # the 8 query heads of kv head 2
                assert torch.equal(lse, clean_lse)
            else:
                hit[sees, 16:24] = True
                assert torch.equal(torch.isnan(lse), hit[..., 0])
            assert bool(same[~hit].all()) and bool(torch.isnan(out[hit]).all())


@pytest.mark.parametrize("fp8", [False, True])
def test_slots_past_two_to_the_31_values(fp8):
    """Rows at the end of a pool of more than 2^31 values: every call writes and reads what it
    does in a small pool, bit for bit, a drafted NaN (its rows are read by address) included."""
    rnd = random.Random(21)
    hq, hk, d, far = 64, 8, 128, 2_200_000
    draft, prior = [40, 9], [500, 1500]
    c = ref.tree_case(rnd, draft, prior, hq, hk, d, fp8=fp8)
    n, S = sum(draft), c["num_slots"]
    parents = [p for t in draft for p in ref.random_parents(rnd, t)]
    drafted = []
    for r, t in enumerate(draft):
        keys = [s + i for s, l in zip(c["seg_starts"][r], c["seg_lens"][r]) for i in range(l)]
        drafted += keys[len(keys) - t:]
    base = far - S
    g = torch.Generator().manual_seed(22)
    new = torch.randn(n, hk, d, generator=g).to(torch.bfloat16).cuda()
    values = new.clone()
    values[7, 3, 50] = math.nan
    pos = torch.randint(0, 1 << 20, (n,), generator=g, dtype=torch.int32).cuda()
    plan = sa.seg_attn_rope_plan(d)

    def steps(case, shift):
        at = torch.tensor(drafted, dtype=torch.int32, device="cuda") + shift
        q = torch.empty_like(case["q"])
        if fp8:
            sa.seg_attn_rope_append_fp8(case["q"], q, new, values, pos, at, plan, case["k_scale"],
                                        case["v_scale"], case["k_pool"], case["v_pool"])
        else:
            sa.seg_attn_rope_append(case["q"], q, new, values, pos, at, plan, case["k_pool"],
                                    case["v_pool"])
        tab = sa.TreeTable.build(draft, [[s + shift for s in x] for x in case["seg_starts"]],
                                 case["seg_lens"], case["num_slots"], hq, hk, d,
                                 parents=parents).to("cuda")
        out, lse = run(dict(case, q=q), tab)
        sa.seg_attn_kv_move(case["k_pool"], case["v_pool"], at[:5].clone(), at[20:25].clone())
        return out, lse

    big = dict(c, num_slots=far)
    for name in ("k_pool", "v_pool"):
        big[name] = torch.empty(far, hk, d, dtype=c[name].dtype, device="cuda")
        big[name][base:] = c[name]
    assert big["k_pool"].numel() > 1 << 31
    o0, l0 = steps(c, 0)
    o1, l1 = steps(big, base)
    assert torch.equal(torch.isnan(o0), torch.isnan(o1)) and bool(torch.isnan(o0).any())
    assert torch.equal(o0.view(torch.int16), o1.view(torch.int16)) and torch.equal(l0, l1)
    kind = torch.uint8 if fp8 else torch.int16
    for name in ("k_pool", "v_pool"):
        assert torch.equal(big[name][base:].view(kind), c[name].view(kind))
    assert sa.seg_attn_take_device_error() == 0


def planted_positions(tab, seg_lens, prior, rnd):
    """Logical keys where a wrong row would come from: one in every K tile (both parities, so
    both softmax groups and every ring stage), the ends of every piece, and both sides of every
    segment boundary at the distances where the copies' boxes of 32, 8 and 4 rows begin."""
    p = tab.desc.pass_
    work = tab.host[p.off_work: p.off_work + 16 * p.num_work].view(-1, 16)
    pos = [i + rnd.randrange(128) for i in range(0, prior, 128)]
    for w in work.tolist():
        pos += [w[3] * 128, w[4] * 128 - 1]
    at = 0
    for l in seg_lens:
        at += l
        pos += [at + x for x in (-33, -32, -9, -8, -5, -4, -1, 0, 3, 4, 7, 8, 31, 32)]
    pos = sorted({x for x in pos if 0 <= x < prior})
    rnd.shuffle(pos)
    return pos


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("draft,hq,hkv,d,factor", [(12, 16, 2, 128, 2.0),   # one query tile
                                                   (40, 8, 1, 128, 2.0),    # two, and one
                                                   (30, 4, 1, 64, 4.0)])
def test_every_row_of_a_long_context_reaches_its_query(fp8, draft, hq, hkv, d, factor):
    """Over 70,000 random keys one V row, or one tile of them, is lost in the sum.  Here every
    (token, head) row looks at one planted key, whose V row is its output: a row read from the
    wrong slot, tile or ring stage shows at full size.  A chain, so the plain prefill has to
    give the same."""
    rnd = random.Random(draft)
    prior = 70000
    c = ref.tree_case(rnd, [draft], [prior], hq, hkv, d, nseg=40, fp8=fp8)
    tab = table(c)
    plain = sa.SegTable.build([draft], c["seg_starts"], c["seg_lens"], c["num_slots"], True,
                              sa.MODE_PREFILL, hq, hkv, d).to("cuda")
    ws = torch.empty(max(16, plain.workspace_bytes), dtype=torch.uint8, device="cuda")
    pos = planted_positions(tab, c["seg_lens"][0], prior, rnd)
    assert tab.desc.pass_.num_work > 30 and len(c["seg_lens"][0]) > 10
    rows = draft * hq // hkv
    keep = c["k_pool"].clone(), c["k_values"].clone()
    for at in range(0, len(pos), rows):
        targets = pos[at:at + rows]
        c["k_pool"].copy_(keep[0])
        c["k_values"].copy_(keep[1])
        ref.plant(c, targets, factor)
        want, want_lse, tol, ltol, top = ref.chain_planted(c, targets)
        assert float(top.min()) > 0.9
        for what in ("tree", "prefill"):
            if what == "tree":
                out, lse = run(c, tab)
            else:
                out, lse = torch.full_like(c["q"], math.nan), torch.empty_like(lse)
                args = (out, lse, plain.device, plain.desc, c["scale"], ws)
                if fp8:
                    sa.seg_attn_prefill_fp8(c["q"], c["k_pool"], c["v_pool"], c["k_scale"],
                                            c["v_scale"], *args)
                else:
                    sa.seg_attn_prefill(c["q"], c["k_pool"], c["v_pool"], *args)
            over = (out.double() - want).abs() / tol
            assert float(over.max()) <= 1.0, (what, at, float(over.max()))
            assert bool(((lse.double() - want_lse).abs() <= ltol).all()), (what, at)
    assert sa.seg_attn_take_device_error() == 0


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("draft,hq,hkv,d", [(12, 16, 2, 128), (40, 8, 1, 128), (30, 4, 1, 64)])
def test_scattered_keys_give_the_bits_of_contiguous_ones(fp8, draft, hq, hkv, d):
    """The same 70,000 keys in 40 segments and in one run of slots: other copies, same arithmetic."""
    rnd = random.Random(draft + 1)
    c = ref.tree_case(rnd, [draft], [70000], hq, hkv, d, nseg=40, fp8=fp8)
    parents = ref.random_parents(rnd, draft)
    slots = ref.request_slots(c, 0)
    flat = dict(c, seg_starts=[[0]], seg_lens=[[slots.numel()]], num_slots=slots.numel(),
                k_pool=c["k_pool"][slots].contiguous(), v_pool=c["v_pool"][slots].contiguous())
    (a, la), (b, lb) = (run(x, table(x, parents=parents)) for x in (c, flat))
    assert bool(torch.isfinite(a).all()) and torch.equal(a, b) and torch.equal(la, lb)


def test_captured_behind_copies_and_a_join_of_streams():
    """The pass is a programmatic dependent of a kernel before it; behind a copy, and behind two
    streams that join, it has to wait for all of them.  Replays with other inputs and another
    table (copied inside the graph) give the eager calls' bits, row moves included."""
    rnd = random.Random(30)
    hq, hk, d = 16, 2, 128
    base = ref.tree_case(rnd, [6, 9], [3000, 700], hq, hk, d)
    forms = [[p for t in base["draft"] for p in ref.random_parents(rnd, t)] for _ in range(4)]
    tabs = [table(base, parents=f) for f in forms]
    assert tabs[0].desc.pass_.num_merge > 0
    assert len({t.desc.table_bytes for t in tabs}) == 1   # the same plan, other masks
    slots = [ref.request_slots(base, r)[-t:].to(torch.int32) for r, t in enumerate(base["draft"])]
    at = torch.cat(slots)
    dev_table = torch.zeros_like(tabs[0].device)
    host_table = torch.empty_like(tabs[0].host, pin_memory=True)
    q, new = torch.empty_like(base["q"]), torch.empty(15, hk, d, dtype=torch.bfloat16, device="cuda")
    host_q, host_new = (torch.empty(t.shape, dtype=t.dtype, pin_memory=True) for t in (q, new))
    kp, vp = base["k_pool"].clone(), base["v_pool"].clone()
    out, lse = torch.empty_like(q), torch.empty(15, hq, device="cuda")
    ws = torch.empty(tabs[0].workspace_bytes, dtype=torch.uint8, device="cuda")
    src, dst = at[[1, 3]].clone(), at[[0, 2]].clone()

    def step(side=None):
        q.copy_(host_q, non_blocking=True)
        if side is not None:
            side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            new.copy_(host_new, non_blocking=True)
            sa.seg_attn_kv_append(new, new, at, kp, vp)
        dev_table.copy_(host_table, non_blocking=True)
        if side is not None:
            torch.cuda.current_stream().wait_stream(side)
        sa.seg_attn_tree(q, kp, vp, out, lse, dev_table, tabs[0].desc, base["scale"], ws)
        sa.seg_attn_kv_move(kp, vp, src, dst)

    def inputs(k):
        g = torch.Generator().manual_seed(100 + k)
        host_q.copy_(torch.randn(q.shape, generator=g))
        host_new.copy_(torch.randn(new.shape, generator=g))
        host_table.copy_(tabs[k].host)

    inputs(0)
    step()
    torch.cuda.synchronize()
    graph, side = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    with torch.cuda.graph(graph):
        step(side)
    for k in range(4):
        inputs(k)
        kp.copy_(base["k_pool"])
        vp.copy_(base["v_pool"])
        step()
        torch.cuda.synchronize()
        want = [x.clone() for x in (out, lse, kp, vp)]
        kp.copy_(base["k_pool"])
        vp.copy_(base["v_pool"])
        out.fill_(math.nan)
        lse.fill_(math.nan)
        torch.cuda.synchronize()
        graph.replay()
        graph.replay()   # twice in a row: the second call's pass behind the first one's move
        torch.cuda.synchronize()
        for a, b in zip((out, lse), want):
            assert torch.equal(a, b) and bool(torch.isfinite(a).all())
        for a, b in zip((kp, vp), want[2:]):
            assert torch.equal(a.view(torch.int16), b.view(torch.int16))
        c = dict(base, q=q)
        if k == 3:   # and they are right, not only alike: the cache before its rows moved
            kv = base["k_pool"].clone(), base["v_pool"].clone()
            for x in kv:
                x[at.long()] = new
            ref.check_tree(out, lse, ref.tree(q, kv[0], kv[1], c["draft"],
                                              ref.visible(c["draft"], parents=forms[k]),
                                              c["seg_starts"], c["seg_lens"], c["scale"]))
    assert sa.seg_attn_take_device_error() == 0
