"""Calls of the serving operators that their declarations allow, at the edges of what they hold.

Plain forms and tolerances are those of test_serving_gpu."""
import math
from fractions import Fraction

import pytest
import torch

from gqa_canvas_attention_gb300 import binding as B
from test_serving_gpu import TYPES, _lib, check_attention, gen, plain_attention  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("hd", [64, 128, 256])
@pytest.mark.parametrize("Bn,T", [(1, 1), (1, 300), (3, 140)])
def test_no_keys(Bn, T, hd):
    """K and V of no rows: every row sees nothing and is 0; rows behind q_len stay."""
    q = torch.randn(Bn, T, 4, hd, generator=gen(T), device="cuda").half()
    none = torch.zeros(Bn, 0, 2, hd, dtype=torch.float16, device="cuda")
    plan = B.WindowPlan(4, 2, hd, Bn, T, 0)
    for lens in (None, [T // 2] * Bn):
        out = torch.full_like(q, 3.0)
        q_len = None if lens is None else torch.tensor(lens, dtype=torch.int32, device="cuda")
        plan.attend(q, none, none, q_len, right=0, out=out)
        n = T if lens is None else T // 2
        assert not out[:, :n].any() and (out[:, n:] == 3.0).all()
    assert plan.sync_status() == B.DG_OK


@pytest.mark.parametrize("dt", ["f16", "bf16"])
@pytest.mark.parametrize("hd", [64, 128, 256])
@pytest.mark.parametrize("T,S", [(1, 300), (3, 4000), (140, 400), (140, 4000)])
def test_scores_of_minus_infinity(T, S, hd, dt):
    """Such keys have no weight, and a row that sees nothing else is 0."""
    g = gen(T + S)
    nh, nkv, left = 4, 2, 20
    q = torch.randn(1, T, nh, hd, generator=g, device="cuda").to(TYPES[dt])
    q[..., 3] = 1
    k = torch.randn(1, S, nkv, hd, generator=g, device="cuda").to(TYPES[dt])
    v = torch.randn(1, S, nkv, hd, generator=g, device="cuda").to(TYPES[dt])
    plan = B.WindowPlan(nh, nkv, hd, 1, T, S)
    k[:, S - left - 1:, 0, 3] = -float("inf")                # the last row of head 0 sees nothing else
    out = plan.attend(q, k, v, left=left, right=0, scale=hd ** -0.5)
    some = k.clone()
    some[:, S - left - 1:, 0, 3] = -60000.0                  # as good as that for rows that see another key
    want, tol = plain_attention(q, some, v, None, None, left, 0, 0, hd ** -0.5, torch.zeros_like(out))
    want[:, -1, :2], tol[:, -1, :2] = 0, 0
    check_attention(out, want, tol, "window")
    k[:, :, 0, 3] = -float("inf")                            # all keys of head 0, in each partition
    out = plan.attend(q, k, v, scale=hd ** -0.5)
    assert not out[:, :, :2].any() and torch.isfinite(out).all()
    assert plan.sync_status() == B.DG_OK


def stored(plan_args, seed, dt):
    """A 4-bit cache of random rows, and its values."""
    Bn, S, nkv, hd = plan_args
    cache = B.Kv4Cache(Bn, nkv, S, hd)
    x = torch.randn(2, Bn, S, nkv, hd, generator=gen(seed), device="cuda").to(TYPES[dt])
    k, v = torch.zeros_like(x[0]), torch.zeros_like(x[1])
    cache.append(x[0], x[1], torch.zeros(Bn, dtype=torch.int32, device="cuda"), k_out=k, v_out=v)
    return cache, k, v


@pytest.mark.parametrize("dt", ["f16", "bf16"])
@pytest.mark.parametrize("T,S,hd", [(1, 700, 128), (5, 3000, 64), (140, 400, 64), (140, 400, 256), (140, 3000, 128),
                                    (140, 3000, 256)])
def test_not_a_number_in_the_cache(T, S, hd, dt):
    """A block of 16 channels that reads as NaN is in the results of the rows that see it, and in no other."""
    nh, nkv = 4, 2
    cache, k, v = stored((1, S, nkv, hd), T, dt)
    q = torch.randn(1, T, nh, hd, generator=gen(S), device="cuda").to(TYPES[dt])
    plan = B.WindowPlan(nh, nkv, hd, 1, T, S)
    far = S - T // 2 - 1
    cache.v_scale[0, 0, far, 1], v[0, far, 0, 16:32] = 0x7F, float("nan")
    cache.k_scale[0, 1, 3, 0], k[0, 3, 1, :16] = 0x7F, float("nan")
    for left, right, sinks in ((-1, -1, 0), (-1, 0, 0), (30, 0, 2), (30, 0, 6), (30, 4, 0)):
        out = plan.attend_kv4(q, cache, left=left, right=right, sinks=sinks, scale=hd ** -0.5)
        want, tol = plain_attention(q, k, v, None, None, left, right, sinks, hd ** -0.5, torch.zeros_like(out))
        rows = torch.isnan(want).all(-1)                     # a NaN score: the whole row
        some = torch.isnan(want).any(-1) & ~rows
        assert torch.isnan(out[rows]).all() and torch.isnan(out[some][:, 16:32]).all()
        check_attention(out, want, tol, f"left {left} right {right} sinks {sinks}")
    assert plan.sync_status() == B.DG_OK


@pytest.mark.parametrize("kv4", [False, True], ids=["16bit", "4bit"])
def test_not_a_number_costs_little(kv4):
    """A NaN score in every row (and for 4-bit keys a NaN value that every row sees) does not make a call of
    50 us one of 100 ms: the rows' second computation ends at the first NaN, or is not begun."""
    nh, nkv, hd, T, S = 8, 4, 256, 512, 8704
    q = torch.randn(1, T, nh, hd, generator=gen(1), device="cuda").half()
    plan = B.WindowPlan(nh, nkv, hd, 1, T, S)
    cache, k, v = stored((1, S, nkv, hd), 2, "f16")
    for side in ("k", "v") if kv4 else ("k",):
        if kv4:
            (cache.k_scale if side == "k" else cache.v_scale)[0, :, 5, 0] = 0x7F
            call = lambda: plan.attend_kv4(q, cache, scale=hd ** -0.5)
        else:
            k[0, 5, :, 0] = float("nan")
            call = lambda: plan.attend(q, k, v, scale=hd ** -0.5)
        assert torch.isnan(call()).any(-1).all()
        start, end = (torch.cuda.Event(enable_timing=True) for _ in range(2))
        start.record()
        call()
        end.record()
        torch.cuda.synchronize()
        assert start.elapsed_time(end) < 10


def pi():
    """pi to some 60 digits (Machin)."""
    arctan = lambda n: sum(Fraction((-1) ** i, (2 * i + 1) * n ** (2 * i + 1)) for i in range(60))
    return 4 * (4 * arctan(5) - arctan(239))


@pytest.mark.parametrize("theta,scaling,factor", [(16.0, 0, 1.0), (10000.0, 0, 1.0), (1000000.0, B.DG_ROPE_SCALE_LINEAR, 4.0)])
def test_angles_of_far_positions(theta, scaling, factor):
    """cos and sin of p f to fp32, f the frequency that the rope reports, for positions far beyond 32 bits.

    The angle is off by |p| 2^-64 turns and 2^-33 of its rounding to 32 bits, its argument by 2^-25 of a half
    turn, the results by 2 ulp."""
    far = [3, 2 ** 31 + 5, -(2 ** 36) - 1, 2 ** 40 + 12345, 2 ** 44 + 7, -(2 ** 44) + 3]
    rope = B.Rope(64, 8, theta=theta, scaling=scaling, factor=factor)
    x = torch.zeros(1, len(far), 1, 64, device="cuda")
    x[..., :4] = 1                                           # pairs (1, 0)
    y, _ = rope.apply(x, None, torch.tensor([far], device="cuda"))
    f, _ = rope.frequencies()
    two_pi = 2 * pi()
    for n, p in enumerate(far):
        for i in range(4):
            angle = float((Fraction(f[i]) * p) % two_pi)
            tol = 2 * math.pi * (abs(p) * 2.0 ** -64 + 2.0 ** -33 + 2.0 ** -26) + 4 * 2.0 ** -24
            assert abs(float(y[0, n, 0, i]) - math.cos(angle)) <= tol, (p, i)
            assert abs(float(y[0, n, 0, 4 + i]) - math.sin(angle)) <= tol, (p, i)


def test_one_buffer_of_heads_outside_tokens():
    """q, k and v as slices of one [batch, heads, T, hd] buffer: in place, and from one half into the other."""
    Bn, T, nh, nkv, hd = 3, 9, 4, 2, 64
    H = nh + 2 * nkv
    rope = B.Rope(hd)
    buf = torch.randn(Bn, H, T, hd, generator=gen(1), device="cuda").bfloat16()
    keep = buf.clone()
    pos = torch.arange(T, device="cuda").repeat(Bn, 1)
    q, k, v = (buf[:, a:b].transpose(1, 2) for a, b in ((0, nh), (nh, nh + nkv), (nh + nkv, H)))
    q0, k0, v0 = (keep[:, a:b].transpose(1, 2) for a, b in ((0, nh), (nh, nh + nkv), (nh + nkv, H)))
    want = rope.qk_norm(q0, k0, v0, pos)
    rope.qk_norm(q, k, v, pos, q_out=q, k_out=k, v_out=v)
    for x, y in zip((q, k, v), want):
        assert torch.equal(x, y)
    rope.apply(k0, None, pos, q_out=q0[:, :, :nkv])
    assert torch.equal(q0[:, :, :nkv], rope.apply(k0, None, pos)[0])
    # the attention's output into other heads of its queries' buffer
    plan = B.WindowPlan(nkv, nkv, hd, Bn, T, T)
    kk, vv = torch.randn(2, Bn, T, nkv, hd, generator=gen(2), device="cuda").bfloat16()
    want = plan.attend(q[:, :, :nkv], kk, vv)
    plan.attend(q[:, :, :nkv], kk, vv, out=q[:, :, nkv:])
    assert torch.equal(q[:, :, nkv:], want)
    with pytest.raises(B.DgAttnError, match="overlaps"):
        plan.attend(q[:, :, :nkv], kk, vv, out=q[:, :, 1:1 + nkv])


@pytest.mark.parametrize("kv4", [False, True], ids=["16bit", "4bit"])
@pytest.mark.parametrize("hd", [64, 128, 256])
@pytest.mark.parametrize("scale", [0.0, -0.0, 1e-36])
def test_scale_0_of_large_products(scale, hd, kv4):
    """Whatever the products are, a scale of 0 (or next to it) makes the weights equal."""
    S, T = 300, 140
    big = 1e32 if kv4 else 1e16
    q = (torch.randn(1, T, 4, hd, generator=gen(hd), device="cuda") * big).bfloat16()
    plan = B.WindowPlan(4, 2, hd, 1, T, S)
    if kv4:
        cache, k, v = stored((1, S, 2, hd), 3, "bf16")
        out = plan.attend_kv4(q, cache, scale=scale)
    else:
        k, v = torch.randn(2, 1, S, 2, hd, generator=gen(4), device="cuda").bfloat16()
        k = (k * big).bfloat16()
        out = plan.attend(q, k, v, scale=scale)
    want, tol = plain_attention(q, k, v, None, None, -1, -1, 0, scale, torch.zeros_like(out))
    check_attention(out, want, tol)
