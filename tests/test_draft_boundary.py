"""Rotary plans, tree tables and argument checks of the drafted-token calls (no GPU)."""
import ctypes
import math
import random

import numpy as np
import pytest
import torch

import segmented_kv_cache_b200 as sa
from segmented_kv_cache_b200 import _build

import draft_reference as ref

S = sa.STATUS


@pytest.fixture(scope="module", autouse=True)
def lib():
    _build.build()
    return sa.load_library()


def code_of(fn):
    with pytest.raises(sa.SegAttnError) as e:
        fn()
    return e.value.code


# ------------------------------------------------------------------------ rotary plans
def turns(desc):
    return [int(desc.turns[i]) for i in range(desc.rotary_dim // 2)]


def same_frequencies(desc, inv_freq):
    """Turn fractions against 64-bit frequencies: a double's 2^-53 and half a unit of 2^-64."""
    for t, w in zip(turns(desc), inv_freq):
        want = w / (2 * math.pi)
        want -= math.floor(want)
        assert abs(t / 2.0 ** 64 - want) <= 4 * 2.0 ** -53 * max(want, 2.0 ** -11)


@pytest.mark.parametrize("rotary", [2, 20, 64, 128, 256])
@pytest.mark.parametrize("base", [10000.0, 500000.0, 1.5])
def test_plain_plan(rotary, base):
    d = sa.seg_attn_rope_plan(rotary, base=base)
    assert d.rotary_dim == rotary and d.layout == 0 and d.amp == 1.0
    same_frequencies(d, ref.plain_freq(rotary, base))
    assert sa.seg_attn_rope_plan(rotary, interleaved=True).layout == 1


def test_scalings():
    r, base, f, L = 64, 10000.0, 8.0, 4096
    w = ref.plain_freq(r, base)
    plan = lambda **kw: sa.seg_attn_rope_plan(r, base=base, scaling=sa.RopeScaling(**kw))
    same_frequencies(plan(kind="none"), w)
    same_frequencies(plan(kind="linear", factor=f), [x / f for x in w])
    same_frequencies(plan(kind="ntk", factor=f), ref.plain_freq(r, base * f ** (r / (r - 2))))
    d = plan(kind="per_pair", factors=[1 + i for i in range(r // 2)])
    same_frequencies(d, [x / (1 + i) for i, x in enumerate(w)])
    # the ends of the blends keep or divide the frequency, and it falls in between
    for kind, high in (("yarn", 32.0), ("wavelength", 4.0)):
        d = plan(kind=kind, factor=f, original_len=L)
        got = [t / 2.0 ** 64 * 2 * math.pi for t in turns(d)]
        ratio = [g / x for g, x in zip(got, w)]
        assert ratio[0] == pytest.approx(1.0) and ratio[-1] == pytest.approx(1 / f)
        assert all(a >= b - 1e-12 for a, b in zip(ratio, ratio[1:]))
        e = plan(kind=kind, factor=f, original_len=L, low=1.0, high=high)
        assert turns(e) == turns(d)
    assert plan(kind="yarn", factor=f, original_len=L).amp == pytest.approx(0.1 * math.log(f) + 1)
    assert plan(kind="yarn", factor=f, original_len=L, amp=1.25).amp == 1.25
    assert plan(kind="linear", factor=f, amp=0.5).amp == 0.5
    # wavelength: k_i at a pair in the blend, by the formula
    d = plan(kind="wavelength", factor=f, original_len=L)
    for i, x in enumerate(w):
        k = min(max((L * x / (2 * math.pi) - 1) / 3, 0), 1)
        assert turns(d)[i] / 2.0 ** 64 * 2 * math.pi == pytest.approx(x * k + x / f * (1 - k), rel=1e-12)


def test_plan_refusals():
    plan = sa.seg_attn_rope_plan
    for r in (0, -2, 3, 258):
        assert code_of(lambda: plan(r)) == S["UNSUPPORTED"]
    for base in (1.0, 0.0, -3.0, math.inf, math.nan):
        assert code_of(lambda: plan(64, base=base)) == S["INVALID_ARG"]
    R = sa.RopeScaling
    for sc in (R("linear", factor=0.0), R("linear", factor=math.nan), R("ntk", factor=-1.0),
               R("yarn", factor=2.0), R("yarn", factor=2.0, original_len=-5),
               R("wavelength", factor=2.0, original_len=100, low=4.0, high=4.0),
               R("wavelength", factor=2.0, original_len=100, low=4.0, high=1.0),
               R("per_pair"), R("per_pair", factors=[1.0] * 31), R("per_pair", factors=[0.0] * 32),
               R("linear", factor=2.0, amp=-1.0), R("linear", factor=2.0, amp=1e300),
               R("yarn", factor=1e-9, original_len=100),
               R("bent")):
        assert code_of(lambda: plan(64, scaling=sc)) == S["INVALID_ARG"], sc
    assert sa.load_library().seg_attn_rope_plan(64, 2, 1e4, None, ctypes.byref(
        sa.seg_attn_rope_desc())) == S["INVALID_ARG"]
    assert sa.load_library().seg_attn_rope_plan(64, 0, 1e4, None, None) == S["INVALID_ARG"]


# ------------------------------------------------------------------------ tree tables
def build(draft, segs, num_slots=4000, hq=8, hkv=2, d=128, **kw):
    return sa.TreeTable.build(draft, [[s for s, _ in r] for r in segs],
                              [[l for _, l in r] for r in segs], num_slots, hq, hkv, d, **kw)


def test_tree_table_refusals():
    ok = [[(0, 10), (100, 20)]]
    build([5], ok)
    assert code_of(lambda: build([5], [[(3995, 10)]])) == S["SEGMENT_OOB"]
    assert code_of(lambda: build([5], [[(-1, 10)]])) == S["SEGMENT_OOB"]
    assert code_of(lambda: build([5], [[(0, 10), (5, 10)]])) == S["SEGMENT_OVERLAP"]
    assert code_of(lambda: build([31], ok)) == S["QLEN_GT_KLEN"]
    assert code_of(lambda: build([-1], ok)) == S["INVALID_ARG"]
    assert code_of(lambda: build([5], [[(0, -1)]])) == S["INVALID_ARG"]
    assert code_of(lambda: build([1025], [[(0, 3000)]])) == S["UNSUPPORTED"]
    build([1024], [[(0, 3000)]])
    for parents in ([0, 0, 1, 2, 3], [-1, 1, 1, 2, 3], [-2, 0, 0, 0, 0], [-1, 5, 0, 0, 0]):
        assert code_of(lambda: build([5], ok, parents=parents)) == S["INVALID_ARG"]
    assert code_of(lambda: build([5], ok, parents=[-1] * 4)) == S["INVALID_ARG"]
    assert code_of(lambda: build([5], ok, mask=[1] * 24)) == S["INVALID_ARG"]
    assert code_of(lambda: build([5], ok, parents=[-1] * 5, mask=[1] * 25)) == S["INVALID_ARG"]
    assert code_of(lambda: build([5], ok, d=96)) == S["UNSUPPORTED"]
    assert code_of(lambda: build([5], ok, hq=6, hkv=2)) == S["UNSUPPORTED"]
    assert code_of(lambda: build([5], ok, hq=6, hkv=4)) == S["INVALID_ARG"]
    assert code_of(lambda: build([5], ok, hq=256, hkv=1)) == S["UNSUPPORTED"]
    assert code_of(lambda: build([5, 5], ok)) == S["INVALID_ARG"]
    assert code_of(lambda: build([1], [[(0, 5)]], num_slots=1 << 31, hq=2, hkv=1)) == S["UNSUPPORTED"]
    # a pool that only just fits the row index, and one past it
    build([1], [[(0, 5)]], num_slots=(1 << 31) // 2 - 1, hq=2, hkv=2)
    assert code_of(lambda: build([1], [[(0, 5)]], num_slots=1 << 30, hq=2, hkv=2)) == S["UNSUPPORTED"]


def test_small_buffer_and_null_desc(lib):
    P = ctypes.c_void_p
    i32 = lambda x: np.array(x, dtype=np.int32)
    dl, sc, ss, sl = i32([3]), i32([1]), i32([0]), i32([200])
    desc = sa.seg_attn_tree_desc()
    args = [1, P(dl.ctypes.data), None, None, P(sc.ctypes.data), P(ss.ctypes.data),
            P(sl.ctypes.data), 300, 4, 2, 64]
    assert lib.seg_attn_build_tree_table(*args, None, 0, None) == S["INVALID_ARG"]
    assert lib.seg_attn_build_tree_table(*args, None, 0, ctypes.byref(desc)) == 0
    need = desc.table_bytes
    buf = np.zeros(need // 4 + 8, dtype=np.int32)
    at = (-buf.ctypes.data) % 16 + buf.ctypes.data
    assert lib.seg_attn_build_tree_table(*args, P(at), need - 4, ctypes.byref(desc)) == \
        S["BUFFER_TOO_SMALL"]
    assert desc.table_bytes == need and lib.seg_attn_tree_workspace_size(ctypes.byref(desc)) == 0
    assert lib.seg_attn_build_tree_table(*args, P(at + 4), need, ctypes.byref(desc)) == S["INVALID_ARG"]
    assert lib.seg_attn_build_tree_table(*args, P(at), need, ctypes.byref(desc)) == 0


@pytest.mark.parametrize("seed", range(6))
@pytest.mark.parametrize("hq,hkv", [(8, 2), (64, 8), (128, 1), (3, 3)])
def test_tree_table_content(seed, hq, hkv):
    rnd = random.Random(seed)
    B = rnd.randint(1, 6)
    draft = [rnd.choice([0, 1, 2, 31, 32, 33, 70, 300]) for _ in range(B)]
    prior = [rnd.choice([0, 1, 127, 128, 129, 3000]) for _ in range(B)]
    c = ref.tree_case(rnd, draft, prior, hq, hkv, 64, device="cpu")
    form = seed % 3
    kw = {}
    if form == 0:
        kw = dict(parents=[p for t in draft for p in ref.random_parents(rnd, t)])
    elif form == 1:
        kw = dict(mask=[rnd.random() < 0.3 for _ in range(sum(t * t for t in draft))])
    tab = sa.TreeTable.build(draft, c["seg_starts"], c["seg_lens"], c["num_slots"], hq, hkv, 64, **kw)
    vis = ref.visible(draft, **kw)
    d, p, host = tab.desc, tab.desc.pass_, tab.host
    slot = host[d.off_draft_slot: d.off_draft_slot + sum(draft)].tolist()
    G = hq // hkv
    qpt = 128 // G
    work = host[p.off_work: p.off_work + 16 * p.num_work].view(-1, 16).tolist()
    merge = host[p.off_merge: p.off_merge + 8 * p.num_merge].view(-1, 8).tolist()
    items = {}
    for w in work:
        items.setdefault((w[0], w[1], w[2]), []).append(w)
    slots_used, at = [], 0
    for r, t in enumerate(draft):
        keys = [s + i for s, l in zip(c["seg_starts"][r], c["seg_lens"][r]) for i in range(l)]
        assert slot[at:at + t] == keys[prior[r]:]
        tiles, nw = (len(keys) + 127) // 128, (t + 31) // 32
        for q0 in range(0, t, 2 * qpt):
            for g in range(hkv):
                got = sorted(items.pop((r, g, q0)), key=lambda w: w[3])
                # the item's pieces cover all of its K tiles
                assert got[0][3] == 0 and got[-1][4] == tiles
                assert all(x[4] == y[3] for x, y in zip(got, got[1:]))
                if len(got) == 1:
                    assert got[0][5] == -1
                else:
                    row = [m for m in merge if m[:3] == [r, g, q0]]
                    assert len(row) == 1 and row[0][4] == len(got)
                    assert [w[5] for w in got] == [row[0][3] + i for i in range(len(got))]
                    slots_used += [w[5] for w in got]
                for w in got:
                    assert w[8:11] == [at, t, len(keys)]
                    m0 = (w[13] & 0xffffffff) | (w[14] << 32)
                    bits = [x & 0xffffffff for x in host[m0:m0 + t * nw].tolist()]
                    for i in range(t):
                        row_bits = bits[i * nw:(i + 1) * nw]
                        assert [bool(row_bits[j >> 5] >> (j & 31) & 1) for j in range(nw * 32)] == \
                            vis[r][i].tolist() + [False] * (nw * 32 - t)
        at += t
    assert not items and sorted(slots_used) == list(range(p.num_parts))
    assert p.num_parts == 0 or tab.workspace_bytes >= p.num_parts * 256 * (64 + 1) * 4


def test_empty_batches():
    tab = sa.TreeTable.build([], [], [], 10, 4, 2, 64)
    assert tab.desc.pass_.total_q == 0 and tab.workspace_bytes == 0
    tab = build([0, 0], [[(0, 10)], []])
    assert tab.desc.pass_.num_work == 0


# ------------------------------------------------------------------------ call refusals
def test_compute_refusals_before_any_launch(lib):
    """Every bad argument is answered on the host (fake addresses: nothing is launched)."""
    A, U = ctypes.c_void_p(1 << 20), ctypes.c_void_p((1 << 20) + 1)
    rope = sa.seg_attn_rope_plan(64)
    R = ctypes.byref(rope)
    f = lib.seg_attn_rope
    I = S["INVALID_ARG"]
    assert f(None, 512, A, 512, A, 2, 4, 128, R, 0, None) == I
    assert f(A, 512, None, 512, A, 2, 4, 128, R, 0, None) == I
    assert f(U, 512, A, 512, A, 2, 4, 128, R, 0, None) == I
    assert f(A, 512, A, 512, None, 2, 4, 128, R, 0, None) == I
    assert f(A, 511, A, 512, A, 2, 4, 128, R, 0, None) == I
    assert f(A, 512, A, 0, A, 2, 4, 128, R, 0, None) == I
    assert f(A, 512, A, 512, A, -1, 4, 128, R, 0, None) == I
    assert f(A, 512, A, 512, A, 2, 0, 128, R, 0, None) == I
    assert f(A, 512, A, 512, A, 2, 4, 62, R, 0, None) == I
    assert f(A, 512, A, 512, A, 2, 4, 128, R, 2, None) == I
    assert f(A, 512, A, 512, A, 2, 4, 128, None, 0, None) == I
    assert f(A, 512, A, 512, A, 2, 4, 128, ctypes.byref(sa.seg_attn_rope_desc()), 0, None) == I
    assert f(A, 1 << 20, A, 1 << 20, A, 2, 4, 8192, R, 0, None) == S["UNSUPPORTED"]
    assert f(None, 0, None, 0, None, 0, 4, 128, R, 0, None) == 0

    def append(q=A, qo=A, k=A, v=A, pos=A, slots=A, n=2, hq=4, hk=2, d=128, kp=A, vp=A, S_=10,
               st=(512, 512, 256, 256)):
        return lib.seg_attn_rope_append(q, st[0], qo, st[1], k, st[2], v, st[3], pos, slots, n, hq,
                                        hk, d, R, kp, vp, S_, None)
    for kw in (dict(q=None), dict(qo=None), dict(k=None), dict(v=None), dict(pos=None),
               dict(slots=None), dict(kp=None), dict(vp=None), dict(n=-1), dict(hq=-1), dict(hk=0),
               dict(S_=-1), dict(d=32), dict(st=(511, 512, 256, 256)), dict(st=(512, 512, 255, 256)),
               dict(st=(512, 512, 256, 0)), dict(slots=U)):
        assert append(**kw) == I, kw
    assert append(n=0, q=None, k=None) == 0
    assert lib.seg_attn_rope_append_fp8(A, 512, A, 512, A, 256, A, 256, A, A, 2, 4, 2, 128, R, None, A,
                                        A, A, 10, None) == I

    g = lib.seg_attn_kv_move
    assert g(None, A, A, A, 3, None, 0, 2, 64, 2, 10, None) == I
    assert g(A, U, A, A, 3, None, 0, 2, 64, 2, 10, None) == I
    assert g(A, A, None, A, 3, None, 0, 2, 64, 2, 10, None) == I
    assert g(A, A, A, U, 3, None, 0, 2, 64, 2, 10, None) == I
    assert g(A, A, A, A, -1, None, 0, 2, 64, 2, 10, None) == I
    assert g(A, A, A, A, 3, A, -1, 2, 64, 2, 10, None) == I
    assert g(A, A, A, A, 3, None, 0, 2, 64, 4, 10, None) == I
    assert g(A, A, A, A, 3, None, 0, 0, 64, 2, 10, None) == I
    assert g(A, A, A, A, 3, None, 0, 2, 64, 2, -1, None) == I
    assert g(A, A, A, A, 3, None, 0, 1, 12, 2, 10, None) == S["UNSUPPORTED"]
    assert g(A, A, A, A, 0, None, 0, 2, 64, 2, 10, None) == 0
    assert g(A, A, A, A, 3, A, 0, 2, 64, 2, 10, None) == 0

    tab = build([3], [[(0, 500)]])
    D = ctypes.byref(tab.desc)
    h = lib.seg_attn_tree
    assert tab.workspace_bytes > 0
    ws = tab.workspace_bytes
    assert h(None, A, A, A, A, A, D, 0.1, A, ws, None) == I
    assert h(A, None, A, A, A, A, D, 0.1, A, ws, None) == I
    assert h(A, A, A, U, A, A, D, 0.1, A, ws, None) == I
    assert h(A, A, A, A, U, A, D, 0.1, A, ws, None) == I
    assert h(A, A, A, A, A, None, D, 0.1, A, ws, None) == I
    assert h(A, A, A, A, A, A, None, 0.1, A, ws, None) == I
    for s in (0.0, -1.0, math.inf, math.nan):
        assert h(A, A, A, A, A, A, D, s, A, ws, None) == I
    assert h(A, A, A, A, A, A, D, 0.1, None, 0, None) == S["WORKSPACE"]
    assert h(A, A, A, A, A, A, D, 0.1, A, ws - 1, None) == S["WORKSPACE"]
    assert h(A, A, A, A, A, A, D, 0.1, U, ws, None) == S["WORKSPACE"]
    assert lib.seg_attn_tree_fp8(A, A, A, None, A, A, A, A, D, 0.1, A, ws, None) == I
    bad = sa.seg_attn_tree_desc.from_buffer_copy(tab.desc)
    bad.version = 99
    assert h(A, A, A, A, A, A, ctypes.byref(bad), 0.1, A, ws, None) == I
    # the plain calls do not take the pass inside a tree table for one of theirs
    assert lib.seg_attn_prefill(A, A, A, A, A, A, ctypes.byref(tab.desc.pass_), 0.1, A, ws, None) == I
    empty = build([0], [[(0, 5)]])
    assert h(None, None, None, None, None, None, ctypes.byref(empty.desc), 0.1, None, 0, None) == 0


def test_binding_checks_dtypes_shapes_and_devices():
    """The Python calls refuse CPU tensors (and say what they want)."""
    x = torch.zeros(2, 4, 128, dtype=torch.bfloat16)
    pos = torch.zeros(2, dtype=torch.int32)
    rope = sa.seg_attn_rope_plan(64)
    pool = torch.zeros(8, 4, 128, dtype=torch.bfloat16)
    assert code_of(lambda: sa.seg_attn_rope(x, x, pos, rope)) == S["INVALID_ARG"]
    assert code_of(lambda: sa.seg_attn_rope_append(x, x, x, x, pos, pos, rope, pool, pool)) == \
        S["INVALID_ARG"]
    assert code_of(lambda: sa.seg_attn_kv_move(pool, pool, pos, pos)) == S["INVALID_ARG"]
    tab = build([2], [[(0, 5)]], num_slots=8, hq=4, hkv=4)
    assert code_of(lambda: sa.seg_attn_tree(x, pool, pool, x, None, tab.host, tab.desc, 0.1)) == \
        S["INVALID_ARG"]


def test_in_place_needs_one_stride(lib):
    """x and out at one address with different token strides would read rows already written."""
    A, B = ctypes.c_void_p(1 << 20), ctypes.c_void_p(1 << 24)
    R = ctypes.byref(sa.seg_attn_rope_plan(64))
    I = S["INVALID_ARG"]
    for x, y in ((512, 768), (768, 512)):
        assert lib.seg_attn_rope(A, x, A, y, B, 2, 4, 128, R, 0, None) == I
        assert lib.seg_attn_rope_append(A, x, A, y, B, 256, B, 256, B, B, 2, 4, 2, 128, R, B, B, 10,
                                        None) == I
        assert lib.seg_attn_rope_append_fp8(A, x, A, y, B, 256, B, 256, B, B, 2, 4, 2, 128, R, B, B, B,
                                            B, 10, None) == I
    # no rows: nothing to refuse
    assert lib.seg_attn_rope(A, 512, A, 768, B, 0, 4, 128, R, 0, None) == 0


def test_sizes_follow_a_refilled_descriptor(lib, monkeypatch):
    """The binding checks tensors against the descriptor as it is now: refilled through the C
    entry for a larger table, the smaller table's tensors are refused and the larger one's pass
    (the call itself is replaced: nothing is launched)."""
    P = ctypes.c_void_p
    i32 = lambda x: np.array(x, dtype=np.int32)
    desc, called = sa.seg_attn_tree_desc(), []
    monkeypatch.setattr(sa, "_cuda_device", lambda fn, name, t, dim: -1)
    monkeypatch.setattr(sa, "_invoke", lambda fn, dev, stream, args: called.append(fn))

    def fill(draft, keys, slots, hq, hk, d):
        dl, sc, ss, sl = i32([draft]), i32([1]), i32([0]), i32([keys])
        args = [1, P(dl.ctypes.data), None, None, P(sc.ctypes.data), P(ss.ctypes.data),
                P(sl.ctypes.data), slots, hq, hk, d]
        assert lib.seg_attn_build_tree_table(*args, None, 0, ctypes.byref(desc)) == 0
        bf = lambda *s: torch.zeros(*s, dtype=torch.bfloat16)
        return dict(q=bf(draft, hq, d), k_pool=bf(slots, hk, d), v_pool=bf(slots, hk, d),
                    out=bf(draft, hq, d), lse=torch.zeros(draft, hq), desc=desc, softmax_scale=0.1,
                    dev_table=torch.zeros(desc.table_bytes // 4, dtype=torch.int32))

    small = fill(3, 40, 50, 4, 2, 64)
    sa.seg_attn_tree(**small)
    large = fill(9, 400, 500, 8, 4, 128)
    sa.seg_attn_tree(**large)
    assert len(called) == 2
    for name in ("q", "k_pool", "v_pool", "out", "lse", "dev_table"):
        assert code_of(lambda: sa.seg_attn_tree(**{**large, name: small[name]})) == S["INVALID_ARG"], name
    scales = lambda n: dict(k_scale=torch.ones(n), v_scale=torch.ones(n))
    codes = {k: large[k].view(torch.uint8)[..., :128] for k in ("k_pool", "v_pool")}
    codes = {k: v.contiguous() for k, v in codes.items()}
    sa.seg_attn_tree_fp8(**{**large, **codes, **scales(4)})
    assert code_of(lambda: sa.seg_attn_tree_fp8(**{**large, **codes, **scales(2)})) == S["INVALID_ARG"]
    assert len(called) == 3


@pytest.mark.parametrize("fp8", [False, True])
def test_planted_keys_show_a_wrong_tile(fp8):
    """The long-context check on the oracle alone: V rows of one K tile taken from another owned
    tile leave the bounds in every row that looks into that tile, and in no other."""
    rnd = random.Random(3)
    draft, prior = 6, 4000
    c = ref.tree_case(rnd, [draft], [prior], 8, 1, 128, fp8=fp8, device="cpu")
    targets = rnd.sample(range(prior), draft * 8)
    targets[:4] = [1280, 1290, 1407, 1408]
    ref.plant(c, targets, 2.0)
    want, _, tol, _, top = ref.chain_planted(c, targets)
    assert float(top.min()) > 0.9
    slots = ref.request_slots(c, 0)
    c["v_values"][slots[1280:1408]] = c["v_values"][slots[256:384]].clone()
    got = ref.chain_planted(c, targets)[0]
    bad = ((got - want).abs() > tol).any(-1).flatten()
    assert bad.tolist() == [1280 <= t < 1408 for t in targets]
