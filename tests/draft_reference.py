"""Plain 64-bit forms of the rotary and drafted-token operators, and their error bounds."""
from __future__ import annotations

import math

import numpy as np
import torch

from segmented_kv_cache_b200 import synth

BF16_HALF = torch.finfo(torch.bfloat16).eps / 2   # half a step relative to the value
E4M3_HALF = 2.0 ** -4


def rope_angles(positions, inv_freq):
    return positions.double().cpu()[:, None] * torch.as_tensor(inv_freq, dtype=torch.float64)


def plain_freq(rotary, base=10000.0):
    return [base ** (-2.0 * i / rotary) for i in range(rotary // 2)]


def rope(x, positions, inv_freq, interleaved=False, amp=1.0, backward=False):
    """x [n, heads, d] -> (64-bit rotated rows, |x0| + |x1| of each value's pair)."""
    x = x.detach().double().cpu()
    r = 2 * len(inv_freq)
    a = rope_angles(positions, inv_freq)[:, None]
    c, s = amp * torch.cos(a), amp * torch.sin(a) * (-1.0 if backward else 1.0)
    i0 = torch.arange(0, r, 2) if interleaved else torch.arange(r // 2)
    i1 = i0 + (1 if interleaved else r // 2)
    y, mag = x.clone(), torch.zeros_like(x)
    y[..., i0] = x[..., i0] * c - x[..., i1] * s
    y[..., i1] = x[..., i1] * c + x[..., i0] * s
    mag[..., i0] = mag[..., i1] = x[..., i0].abs() + x[..., i1].abs()
    return y, mag


def rope_tolerance(y, mag, amp=1.0):
    """One rounding to bf16, and in fp32: the angle (2^-24 half turns, i.e. 1.9e-7), cosine and
    sine (2 ulp), their product with amp, two products and a sum: under 8 roundings of 2^-24
    of |x0| + |x1|, so 1e-6 covers both."""
    return BF16_HALF * y.abs() * (1 + 1e-3) + 1e-6 * amp * mag


def visible(draft, parents=None, mask=None):
    """Per request [T, T] bool: what each drafted token sees of the drafts."""
    out, at, at2 = [], 0, 0
    for t in draft:
        m = np.zeros((t, t), dtype=bool)
        if mask is not None:
            m[:] = np.asarray(mask[at2:at2 + t * t]).reshape(t, t) != 0
        else:
            for i in range(t):
                j = i
                while j >= 0:
                    m[i, j] = True
                    j = parents[at + j] if parents is not None else j - 1
        out.append(m)
        at, at2 = at + t, at2 + t * t
    return out


def tree(q, k_pool, v_pool, draft, vis, seg_starts, seg_lens, scale):
    """(out, lse, sum of p |v|) in 64 bits; rows that see a NaN or infinity get what IEEE gives,
    rows that do not are computed without it."""
    q, dev = q.double(), q.device
    hq, d = q.shape[1], q.shape[2]
    hk = k_pool.shape[1]
    g = hq // hk
    outs, lses, mags, at = [], [], [], 0
    for r, t in enumerate(draft):
        slots = torch.tensor([s + i for s, l in zip(seg_starts[r], seg_lens[r]) for i in range(l)],
                             dtype=torch.long, device=dev)
        n = slots.numel()
        k, v = k_pool[slots].double(), v_pool[slots].double()
        see = torch.ones(t, n, dtype=torch.bool)
        if t:
            see[:, n - t:] = torch.from_numpy(vis[r])
        see = see.to(dev)
        qr = q[at:at + t].view(t, hk, g, d)
        at += t
        s = torch.einsum("thgd,khd->thgk", qr, k) * scale
        s = s.masked_fill(~see[:, None, None], -math.inf)
        lse = torch.logsumexp(s, -1) if n else torch.full((t, hk, g), -math.inf, dtype=torch.float64,
                                                          device=dev)
        p = torch.exp(s - torch.where(lse == -math.inf, torch.zeros_like(lse), lse)[..., None])
        good = torch.isfinite(v)
        v0 = torch.where(good, v, torch.zeros_like(v))
        o = torch.einsum("thgk,khd->thgd", p, v0)
        mag = torch.einsum("thgk,khd->thgd", p, v0.abs())
        if not bool(good.all()):
            hit = torch.einsum("tk,khd->thd", see.double(), (~good).double()) > 0
            o = torch.where(hit[:, :, None], torch.full_like(o, math.nan), o)
        outs.append(o.reshape(t, hq, d))
        mags.append(mag.reshape(t, hq, d))
        lses.append(lse.reshape(t, hq))
    cat = lambda x, *s: torch.cat(x) if x else torch.zeros(0, *s, dtype=torch.float64, device=dev)
    return cat(outs, hq, d).cpu(), cat(lses, hq).cpu(), cat(mags, hq, d).cpu()


def check_tree(out, lse, ref, what=""):
    """Bounds: out rounds to bf16 once; a weight rounds to bf16 (f16 over an E4M3 cache), so a row
    is off by at most half a step of sum p |v| more; a score is a sum of <= 128 exact products in
    fp32, off by under 128 * 2^-24 of sum |q k| scale (below 20 for these inputs), i.e. 1.6e-4,
    which moves each weight and their sum by that much: 4e-4 of sum p |v| with the exponentials."""
    ro, rl, mag = ref
    o, l = out.detach().double().cpu(), lse.detach().double().cpu()
    bad = torch.isnan(ro)
    assert torch.equal(torch.isnan(o), bad), f"{what}: NaN rows differ"
    tol = BF16_HALF * ro.abs() + (BF16_HALF + 4e-4) * mag + 1e-30
    over = ((o - ro).abs() / tol)[~bad]
    assert not over.numel() or float(over.max()) <= 1.0, f"{what}: out {float(over.max())} of bound"
    nan = torch.isnan(rl)
    assert torch.equal(torch.isnan(l), nan), f"{what}: NaN lse rows differ"
    inf = torch.isinf(rl)
    assert torch.equal(l[inf], rl[inf]), f"{what}: infinite lse rows differ"
    fin = ~(nan | inf)
    if bool(fin.any()):
        assert float((l[fin] - rl[fin]).abs().max()) <= 3e-4, f"{what}: lse"


def random_parents(rnd, t):
    return [-1 if i == 0 or rnd.random() < 0.1 else rnd.randrange(max(0, i - 6), i) for i in range(t)]


def tree_case(rnd, draft, prior, hq, hkv, d, nseg=3, fp8=False, device="cuda", extra=37):
    """Seeded inputs: NaN in every slot that no request owns."""
    segs = []
    for t, p in zip(draft, prior):
        n = t + p
        cuts = sorted(rnd.randint(0, n) for _ in range(rnd.randint(1, nseg) - 1))
        segs.append([b - a for a, b in zip([0] + cuts, cuts + [n])])
    flat = [x for s in segs for x in s]
    slots = sum(flat) + extra
    g = torch.Generator().manual_seed(rnd.randrange(1 << 30))
    starts = iter(synth.place_segments(flat, slots, g))
    seg_starts = [[next(starts) for _ in s] for s in segs]
    live = torch.zeros(slots, dtype=torch.bool)
    for ss, ll in zip(seg_starts, segs):
        for s, l in zip(ss, ll):
            live[s:s + l] = True
    n = int(live.sum())
    c = dict(draft=list(draft), seg_starts=seg_starts, seg_lens=segs, num_slots=slots,
             scale=1 / math.sqrt(d), fp8=fp8)
    c["q"] = torch.randn(sum(draft), hq, d, generator=g).to(torch.bfloat16).to(device)
    for name in ("k", "v"):
        x = torch.full((slots, hkv, d), math.nan)
        x[live] = torch.randn(n, hkv, d, generator=g)
        if fp8:
            scale = (torch.rand(hkv, generator=g) + 0.5) / 16
            codes = (x / scale[:, None]).clamp(-448, 448).to(torch.float8_e4m3fn)
            c[name + "_scale"] = scale.to(device)
            c[name + "_pool"] = codes.view(torch.uint8).to(device)
            c[name + "_values"] = (codes.double() * scale.double()[:, None]).to(device)
        else:
            c[name + "_pool"] = x.to(torch.bfloat16).to(device)
            c[name + "_values"] = c[name + "_pool"]
    return c


def request_slots(c, r, device=None):
    """Pool slots of request r's keys, in logical order."""
    runs = [torch.arange(s, s + l) for s, l in zip(c["seg_starts"][r], c["seg_lens"][r])]
    return torch.cat(runs).to(device if device is not None else c["q"].device)


def plant(c, targets, factor):
    """Make row (token i, head h) of a one-request case look at one key: the key of logical
    position targets[i * group + h % group] becomes `factor` times the row's query, which
    outweighs all random keys together.  Changes k_pool and k_values in place."""
    t, hq, _ = c["q"].shape
    hkv = c["k_pool"].shape[1]
    group = hq // hkv
    slots = request_slots(c, 0)[torch.tensor(targets, device=c["q"].device)]
    for g in range(hkv):
        rows = c["q"][:, g * group:(g + 1) * group].reshape(t * group, -1)[:len(targets)].float() * factor
        if c["fp8"]:
            scale = c["k_scale"][g]
            codes = (rows / scale).clamp(-448, 448).to(torch.float8_e4m3fn)
            c["k_pool"][slots, g] = codes.view(torch.uint8)
            c["k_values"][slots, g] = codes.double() * scale.double()
        else:
            c["k_pool"][slots, g] = rows.to(torch.bfloat16)   # k_values is the pool


def chain_planted(c, targets):
    """64-bit (out, lse, bound of out, bound of lse, weight of each row's planted key) of a
    one-request chain of drafts after `plant`.

    Bounds: a score is a sum of <= 128 exact products in fp32, off by e = 128 * 2^-24 of the
    largest sum of |q k| scale, which moves a weight and the sum of weights by e each; an
    accumulator rounds once per 16 keys, by 2^-23 of sum p |v| at most (the same for the sum
    of weights); a weight is rounded to bf16 (2^-8) or f16 (2^-11), and one that f16 holds as
    a subnormal or zero loses at most itself, all of them at most 1 - the planted key's
    weight; out rounds to bf16 once."""
    q = c["q"].double()
    t, hq, d = q.shape
    hkv = c["k_pool"].shape[1]
    group = hq // hkv
    slots = request_slots(c, 0)
    n = slots.numel()
    prior = n - t
    step = 2.0 ** -11 if c["fp8"] else BF16_HALF
    out, lse, tol, ltol, top = (torch.empty_like(q), q.new_empty(t, hq), torch.empty_like(q),
                                q.new_empty(t, hq), [])
    for g in range(hkv):
        k, v = c["k_values"][slots, g].double(), c["v_values"][slots, g].double()
        qr = q[:, g * group:(g + 1) * group].reshape(t * group, d)
        s = qr @ k.T * c["scale"]
        tok = torch.arange(t * group, device=q.device) // group
        s = s.masked_fill(torch.arange(n, device=q.device)[None] > prior + tok[:, None], -math.inf)
        e = 128 * 2.0 ** -24 * float((qr.abs() @ k.abs().T).max()) * c["scale"]
        sums = 2 * n / 16 * 2.0 ** -23
        l = torch.logsumexp(s, -1)
        p = torch.exp(s - l[:, None])
        o, mag = p @ v, p @ v.abs()
        rows = torch.arange(len(targets), device=q.device)
        w = p[rows, torch.tensor(targets, device=q.device)]
        top.append(w)
        b = BF16_HALF * o.abs() + (step + 2 * e + sums) * mag
        if c["fp8"]:
            b[:len(targets)] += (1 - w)[:, None] * v.abs().max()
        heads = slice(g * group, (g + 1) * group)
        out[:, heads], lse[:, heads] = o.view(t, group, d), l.view(t, group)
        tol[:, heads], ltol[:, heads] = b.view(t, group, d), e + sums + 1e-4
    return out, lse, tol, ltol, torch.cat(top)
