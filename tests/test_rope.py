"""Rotary positions and the rotated append on the GPU against 64-bit forms."""
import math

import pytest
import torch

import segmented_kv_cache_b200 as sa

import draft_reference as ref

pytestmark = pytest.mark.gpu


def rows(g, n, h, d):
    return torch.randn(n, h, d, generator=g).to(torch.bfloat16)


def positions(g, n, far=False):
    hi = (1 << 31) - 1 if far else 5000
    p = torch.randint(0, hi, (n,), generator=g, dtype=torch.int64)
    if far and n > 2:
        p[0], p[1], p[2] = hi, -hi, -1
    return p.to(torch.int32)


def check(out, x, pos, inv, inter, amp=1.0, backward=False, what=""):
    y, mag = ref.rope(x, pos, inv, inter, amp, backward)
    err = (out.double().cpu() - y).abs()
    over = err / (ref.rope_tolerance(y, mag, amp) + 1e-30)
    assert float(over.max()) <= 1.0, (what, float(over.max()))


@pytest.mark.parametrize("n", [1, 2, 37, 513, 3001])
@pytest.mark.parametrize("h,d,r", [(64, 128, 128), (8, 128, 64), (1, 64, 64), (3, 64, 16), (5, 96, 96),
                                   (2, 80, 32), (4, 256, 256), (1, 16, 16)])
@pytest.mark.parametrize("inter", [False, True])
def test_vector_rows(n, h, d, r, inter):
    g = torch.Generator().manual_seed(n * 7 + h + d + r)
    x, pos = rows(g, n, h, d), positions(g, n)
    plan = sa.seg_attn_rope_plan(r, interleaved=inter)
    xd, out = x.cuda(), torch.full_like(x, math.nan, device="cuda")
    sa.seg_attn_rope(xd, out, pos.cuda(), plan)
    check(out, x, pos, ref.plain_freq(r), inter, what="forward")
    assert torch.equal(out[..., r:].cpu().view(torch.int16), x[..., r:].view(torch.int16))
    assert torch.equal(xd.cpu().view(torch.int16), x.view(torch.int16))
    sa.seg_attn_rope(xd, xd, pos.cuda(), plan, backward=True)   # in place
    check(xd, x, pos, ref.plain_freq(r), inter, backward=True, what="backward in place")


@pytest.mark.parametrize("h,d,r", [(3, 128, 20), (2, 66, 66), (1, 7, 6), (5, 40, 2), (4, 100, 96)])
@pytest.mark.parametrize("inter", [False, True])
def test_odd_sizes_take_the_element_kernel(h, d, r, inter):
    g = torch.Generator().manual_seed(h + d + r)
    n = 131
    x, pos = rows(g, n, h, d), positions(g, n)
    plan = sa.seg_attn_rope_plan(r, interleaved=inter)
    out = torch.full_like(x, math.nan, device="cuda")
    sa.seg_attn_rope(x.cuda(), out, pos.cuda(), plan)
    check(out, x, pos, ref.plain_freq(r), inter)
    assert torch.equal(out[..., r:].cpu().view(torch.int16), x[..., r:].view(torch.int16))


@pytest.mark.parametrize("inter", [False, True])
def test_far_positions_keep_their_angle(inter):
    g = torch.Generator().manual_seed(3)
    n, h, d = 257, 2, 128
    x, pos = rows(g, n, h, d), positions(g, n, far=True)
    plan = sa.seg_attn_rope_plan(d, interleaved=inter)
    out = torch.empty_like(x, device="cuda")
    sa.seg_attn_rope(x.cuda(), out, pos.cuda(), plan)
    # a position near 2^31 times a 64-bit frequency is itself off by 2^31 * 2^-53 radians
    y, mag = ref.rope(x, pos, ref.plain_freq(d), inter)
    err = (out.double().cpu() - y).abs()
    assert float((err / (ref.rope_tolerance(y, mag) + 2.0 ** -20 * mag)).max()) <= 1.0


def test_strided_rows_alignment_and_amplitude():
    """Parts of one projection; a start that is not 16-byte aligned; an odd stride; amplitude."""
    g = torch.Generator().manual_seed(4)
    n, hq, hk, d = 77, 6, 2, 64
    qkv = rows(g, n, hq + 2 * hk, d)
    pos = positions(g, n)
    plan = sa.seg_attn_rope_plan(d, scaling=sa.RopeScaling("linear", factor=4.0, amp=1.5))
    inv = [w / 4 for w in ref.plain_freq(d)]
    dev = qkv.cuda()
    part = dev[:, hq:hq + hk]
    out = torch.empty(n, hk, d, dtype=torch.bfloat16, device="cuda")
    sa.seg_attn_rope(part, out, pos.cuda(), plan)
    check(out, qkv[:, hq:hq + hk], pos, inv, False, amp=1.5)
    sa.seg_attn_rope(part, part, pos.cuda(), plan)   # in place inside the projection
    check(dev[:, hq:hq + hk], qkv[:, hq:hq + hk], pos, inv, False, amp=1.5)
    for lo, hi in ((0, hq), (hq + hk, hq + 2 * hk)):
        assert torch.equal(dev[:, lo:hi].cpu(), qkv[:, lo:hi])
    # one element off: 2-byte alignment and an odd token stride
    flat = torch.randn(1 + n * (hk * d + 3), generator=g).to(torch.bfloat16)
    view = lambda t: torch.as_strided(t, (n, hk, d), (hk * d + 3, d, 1), 1)
    out = torch.empty(n, hk, d, dtype=torch.bfloat16, device="cuda")
    sa.seg_attn_rope(view(flat.cuda()), out, pos.cuda(), plan)
    check(out, view(flat), pos, inv, False, amp=1.5)


def test_nan_and_infinity_stay_in_their_pair():
    g = torch.Generator().manual_seed(5)
    x = rows(g, 9, 2, 64)
    x[3, 1, 5], x[4, 0, 40] = math.nan, math.inf
    pos = positions(g, 9)
    out = torch.empty_like(x, device="cuda")
    sa.seg_attn_rope(x.cuda(), out, pos.cuda(), sa.seg_attn_rope_plan(64))
    bad = ~torch.isfinite(out.cpu())
    want = torch.zeros_like(bad)
    want[3, 1, [5, 37]] = True
    want[4, 0, [8, 40]] = True
    assert torch.equal(bad, want)


def test_backward_is_the_gradient():
    """<g, y(x)> differs by <backward(g), dx>: against differences of the 64-bit form, and as
    the exact transpose."""
    g = torch.Generator().manual_seed(6)
    n, h, d, r = 33, 3, 128, 64
    x, gr, pos = rows(g, n, h, d), rows(g, n, h, d), positions(g, n)
    sc = sa.RopeScaling("yarn", factor=4.0, original_len=1024)
    for inter in (False, True):
        plan = sa.seg_attn_rope_plan(r, interleaved=inter, scaling=sc)
        inv = [int(plan.turns[i]) / 2.0 ** 64 * 2 * math.pi for i in range(r // 2)]
        dx = torch.empty_like(x, device="cuda")
        sa.seg_attn_rope(gr.cuda(), dx, pos.cuda(), plan, backward=True)
        check(dx, gr, pos, inv, inter, amp=plan.amp, backward=True)
        f = lambda v: float((ref.rope(v, pos, inv, inter, plan.amp)[0] * gr.double()).sum())
        for _ in range(8):
            step = torch.zeros(n, h, d, dtype=torch.float64)
            i = tuple(int(torch.randint(0, s, (1,), generator=g)) for s in (n, h, d))
            step[i] = 1e-3
            diff = (f(x.double() + step) - f(x.double() - step)) / 2e-3
            # the operator is linear: the difference is exact but for 64-bit rounding of sums
            assert abs(diff - float(dx[i])) <= ref.BF16_HALF * abs(diff) + 1e-4


def test_current_plans_of_every_scaling():
    g = torch.Generator().manual_seed(7)
    x, pos = rows(g, 50, 2, 64), positions(g, 50)
    for sc in (sa.RopeScaling("linear", factor=2.0), sa.RopeScaling("ntk", factor=4.0),
               sa.RopeScaling("yarn", factor=8.0, original_len=512),
               sa.RopeScaling("wavelength", factor=8.0, original_len=512),
               sa.RopeScaling("per_pair", factors=[1.0 + i for i in range(32)])):
        plan = sa.seg_attn_rope_plan(64, scaling=sc)
        inv = [int(plan.turns[i]) / 2.0 ** 64 * 2 * math.pi for i in range(32)]
        out = torch.empty_like(x, device="cuda")
        sa.seg_attn_rope(x.cuda(), out, pos.cuda(), plan)
        check(out, x, pos, inv, False, amp=plan.amp, what=sc.kind)


# ----------------------------------------------------------------------------- append
def append_inputs(seed, n, hq, hk, d, S):
    g = torch.Generator().manual_seed(seed)
    qkv = rows(g, n, hq + 2 * hk, d)
    slots = torch.randperm(S, generator=g)[:n].to(torch.int32)
    return g, qkv, positions(g, n), slots


@pytest.mark.parametrize("n", [1, 3, 130, 1500])
@pytest.mark.parametrize("hq,hk,d,r", [(64, 8, 128, 128), (8, 1, 64, 32), (4, 4, 128, 64),
                                       (2, 2, 64, 20), (3, 1, 96, 96), (0, 2, 64, 64)])
@pytest.mark.parametrize("inter", [False, True])
def test_append(n, hq, hk, d, r, inter):
    S = n + 23
    g, qkv, pos, slots = append_inputs(n + hq, n, hq, hk, d, S)
    pools = [torch.randn(S, hk, d, generator=g).to(torch.bfloat16) for _ in range(2)]
    kp, vp = (p.cuda() for p in pools)
    plan = sa.seg_attn_rope_plan(r, interleaved=inter)
    dev = qkv.cuda()
    q = dev[:, :hq] if hq else None
    q_out = torch.full((n, hq, d), math.nan, dtype=torch.bfloat16, device="cuda") if hq else None
    sa.seg_attn_rope_append(q, q_out, dev[:, hq:hq + hk], dev[:, hq + hk:], pos.cuda(),
                            slots.cuda(), plan, kp, vp)
    inv = ref.plain_freq(r)
    if hq:
        check(q_out, qkv[:, :hq], pos, inv, inter, what="q")
    check(kp[slots.long().cuda()], qkv[:, hq:hq + hk], pos, inv, inter, what="k")
    want = pools[1].clone()
    want[slots.long()] = qkv[:, hq + hk:]
    assert torch.equal(vp.cpu().view(torch.int16), want.view(torch.int16))
    rest = torch.ones(S, dtype=torch.bool)
    rest[slots.long()] = False
    assert torch.equal(kp.cpu()[rest], pools[0][rest])
    assert torch.equal(dev.cpu().view(torch.int16), qkv.view(torch.int16))
    assert sa.seg_attn_take_device_error() == 0


@pytest.mark.parametrize("n", [1, 200])
@pytest.mark.parametrize("hq,hk,d,r", [(64, 8, 128, 128), (4, 2, 64, 32), (2, 2, 64, 20)])
@pytest.mark.parametrize("inter", [False, True])
def test_append_fp8(n, hq, hk, d, r, inter):
    S = n + 9
    g, qkv, pos, slots = append_inputs(n + hq, n, hq, hk, d, S)
    qkv[0, hq, 0], qkv[0, hq + hk, 3] = 300.0, -250.0   # saturate
    ks, vs = (torch.rand(hk, generator=g) + 0.5 for _ in range(2))
    ks, vs = ks / 16, vs / 16
    kp, vp = (torch.full((S, hk, d), 0x55, dtype=torch.uint8, device="cuda") for _ in range(2))
    plan = sa.seg_attn_rope_plan(r, interleaved=inter)
    dev = qkv.cuda()
    q_out = torch.empty(n, hq, d, dtype=torch.bfloat16, device="cuda")
    sa.seg_attn_rope_append_fp8(dev[:, :hq], q_out, dev[:, hq:hq + hk], dev[:, hq + hk:],
                                pos.cuda(), slots.cuda(), plan, ks.cuda(), vs.cuda(), kp, vp)
    inv = ref.plain_freq(r)
    check(q_out, qkv[:, :hq], pos, inv, inter, what="q")
    y, mag = ref.rope(qkv[:, hq:hq + hk], pos, inv, inter)
    y, mag = y / ks.double()[:, None], mag / ks.double()[:, None]
    y = y.clamp(-448, 448)
    got = kp[slots.long().cuda()].cpu().view(torch.float8_e4m3fn).double()
    # half a step of a normal code, of a subnormal one (2^-10), and the fp32 rotation
    tol = ref.E4M3_HALF * y.abs() + 2.0 ** -10 + 2e-6 * mag
    assert float(((got - y).abs() / tol).max()) <= 1.0
    # values are only quantised: the codes of the plain append
    kp2, vp2 = torch.zeros_like(kp), torch.full_like(vp, 0x55)
    v = qkv[:, hq + hk:].contiguous().cuda()
    sa.seg_attn_kv_append_fp8(v, v, slots.cuda(), ks.cuda(), vs.cuda(), kp2, vp2)
    assert torch.equal(vp, vp2)
    assert sa.seg_attn_take_device_error() == 0


@pytest.mark.parametrize("r", [64, 20])
@pytest.mark.parametrize("fp8", [False, True])
def test_append_skips_and_flags_slots_out_of_range(r, fp8):
    S, hk, d = 16, 2, 64
    x = torch.ones(4, hk, d, dtype=torch.bfloat16, device="cuda")
    pos = torch.zeros(4, dtype=torch.int32, device="cuda")
    slots = torch.tensor([3, -1, S, 10], dtype=torch.int32, device="cuda")
    kp = torch.zeros(S, hk, d, dtype=torch.uint8 if fp8 else torch.bfloat16, device="cuda")
    vp, q_out = torch.zeros_like(kp), torch.zeros_like(x)
    plan = sa.seg_attn_rope_plan(r)
    if fp8:
        one = torch.ones(hk, device="cuda")
        sa.seg_attn_rope_append_fp8(x, q_out, x, x, pos, slots, plan, one, one, kp, vp)
    else:
        sa.seg_attn_rope_append(x, q_out, x, x, pos, slots, plan, kp, vp)
    assert sa.seg_attn_take_device_error() == 2
    assert sa.seg_attn_take_device_error() == 0
    for p in (kp, vp):
        assert (p != 0).flatten(1).any(1).nonzero().flatten().tolist() == [3, 10]
    assert torch.equal(q_out, x)   # position 0 turns nothing, and every query row is written


def test_append_then_plain_append_agree_at_position_zero():
    """Angle 0: the rotated append writes seg_attn_kv_append's bits."""
    g = torch.Generator().manual_seed(8)
    n, hk, d, S = 300, 8, 128, 512
    k, v = rows(g, n, hk, d).cuda(), rows(g, n, hk, d).cuda()
    slots = torch.randperm(S, generator=g)[:n].to(torch.int32).cuda()
    a = [torch.zeros(S, hk, d, dtype=torch.bfloat16, device="cuda") for _ in range(4)]
    pos = torch.zeros(n, dtype=torch.int32, device="cuda")
    sa.seg_attn_rope_append(None, None, k, v, pos, slots, sa.seg_attn_rope_plan(d), a[0], a[1])
    sa.seg_attn_kv_append(k, v, slots, a[2], a[3])
    assert torch.equal(a[0], a[2]) and torch.equal(a[1], a[3])


def test_captured_on_another_stream_and_replayed_with_new_inputs():
    g = torch.Generator().manual_seed(9)
    n, hq, hk, d, S = 40, 4, 2, 64, 64
    qkv = rows(g, n, hq + 2 * hk, d).cuda()
    pos, slots = positions(g, n).cuda(), torch.randperm(S, generator=g)[:n].to(torch.int32).cuda()
    kp, vp = (torch.zeros(S, hk, d, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    q_out = torch.empty(n, hq, d, dtype=torch.bfloat16, device="cuda")
    plan = sa.seg_attn_rope_plan(d)
    call = lambda: sa.seg_attn_rope_append(qkv[:, :hq], q_out, qkv[:, hq:hq + hk], qkv[:, hq + hk:],
                                           pos, slots, plan, kp, vp)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        call()
    plan = None   # the plan is taken by value
    for k in range(3):
        fresh = rows(g, n, hq + 2 * hk, d)
        new_pos = positions(g, n)
        qkv.copy_(fresh)
        pos.copy_(new_pos)
        graph.replay()
        torch.cuda.synchronize()
        check(q_out, fresh[:, :hq], new_pos, ref.plain_freq(d), False)
        check(kp[slots.long()], fresh[:, hq:hq + hk], new_pos, ref.plain_freq(d), False)


def test_binding_refuses_wrong_tensors():
    x = torch.zeros(4, 2, 64, dtype=torch.bfloat16, device="cuda")
    pos = torch.zeros(4, dtype=torch.int32, device="cuda")
    plan = sa.seg_attn_rope_plan(64)
    pool = torch.zeros(8, 2, 64, dtype=torch.bfloat16, device="cuda")
    bad = [
        lambda: sa.seg_attn_rope(x.float(), x, pos, plan),
        lambda: sa.seg_attn_rope(x, x[:3], pos, plan),
        lambda: sa.seg_attn_rope(x, x, pos.long(), plan),
        lambda: sa.seg_attn_rope(x, x, pos[:3], plan),
        lambda: sa.seg_attn_rope(x, x, pos.cpu(), plan),
        lambda: sa.seg_attn_rope(x.transpose(0, 1), x.transpose(0, 1), pos[:2], plan),
        lambda: sa.seg_attn_rope(x[:1].expand(4, 2, 64), x, pos, plan),
        lambda: sa.seg_attn_rope_append(x, x, x, x, pos, pos, plan, pool, pool.view(torch.int16)),
        lambda: sa.seg_attn_rope_append(x, x, x, x[:, :1], pos, pos, plan, pool, pool),
        lambda: sa.seg_attn_rope_append(x, x, x, x, pos, pos, plan, pool, pool[:4]),
        lambda: sa.seg_attn_rope_append(x, None, x, x, pos, pos, plan, pool, pool),
        lambda: sa.seg_attn_rope_append_fp8(x, x, x, x, pos, pos, plan, pos, pos, pool, pool),
    ]
    for i, f in enumerate(bad):
        with pytest.raises(sa.SegAttnError) as e:
            f()
        assert e.value.code == sa.STATUS["INVALID_ARG"], i


@pytest.mark.parametrize("r", [64, 20])   # the vector kernel and the element-wise one
@pytest.mark.parametrize("inter", [False, True])
def test_unrotated_codes_are_the_plain_appends(r, inter):
    """Zeros of both signs, infinities, NaN, saturating and tiny values, and scales on both sides
    of the range where the quotient is a corrected product: V rows and the unrotated tail of K
    rows take seg_attn_kv_append_fp8's codes, which are within half a step of the division."""
    g = torch.Generator().manual_seed(10)
    scales = [1 / 16, 0.0371, 1e-17, 1.7e-19, 3e-24, 6e16, 2.3e19, 1e-39]
    n, hk, d = 64, len(scales), 128
    S = n + 5
    s = torch.tensor(scales, dtype=torch.float32)
    kv = (torch.randn(n, 2 * hk, d, generator=g) * s.repeat(2)[:, None] * 60).to(torch.bfloat16)
    tail = torch.tensor([-0.0, 0.0, math.inf, -math.inf, math.nan, 3e38, -3e38, 1e-40, -1e-40,
                         1e-38, -1e-38, 448.0, -448.0])
    for h in range(2 * hk):
        kv[h % n, h, -len(tail):] = tail.to(torch.bfloat16)
        kv[(h + 20) % n, h, -8:] = torch.tensor([-0.0, 0.0] * 4).to(torch.bfloat16)
    k, v = kv[:, :hk].contiguous().cuda(), kv[:, hk:].contiguous().cuda()
    slots = torch.randperm(S, generator=g)[:n].to(torch.int32).cuda()
    pos, sd = positions(g, n).cuda(), s.cuda()
    a = [torch.full((S, hk, d), 0x55, dtype=torch.uint8, device="cuda") for _ in range(4)]
    sa.seg_attn_rope_append_fp8(None, None, k, v, pos, slots, sa.seg_attn_rope_plan(r, interleaved=inter),
                                sd, sd, a[0], a[1])
    sa.seg_attn_kv_append_fp8(k, v, slots, sd, sd, a[2], a[3])
    assert torch.equal(a[1], a[3])
    assert torch.equal(a[0][..., r:], a[2][..., r:])
    got = a[1][slots.long()].cpu()
    x = kv[:, hk:].double() / s.double()[:, None]
    zero = x == 0
    assert bool(zero.any()) and torch.equal(got[zero], torch.where(torch.signbit(x[zero]), 0x80, 0).to(torch.uint8))
    nan = torch.isnan(x)
    assert bool(((got[nan] & 0x7F) == 0x7F).all())
    value = got.view(torch.float8_e4m3fn).double()
    # half a step of a normal code or of a subnormal one
    off = (value - x.clamp(-448, 448)).abs()[~nan]
    assert bool((off <= ref.E4M3_HALF * x[~nan].abs().clamp(max=448) + 2.0 ** -10).all())
    assert sa.seg_attn_take_device_error() == 0
