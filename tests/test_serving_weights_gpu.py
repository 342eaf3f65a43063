"""Weights far below a row's largest: one key that leads thousands of others, as the first tokens do in
a model with sink tokens, with a value of its own.

Tolerances count roundings, against 64 bits.  A score z = scale sum q k is off by dz = 2^-21 scale
sum |q k| (hd products summed in fp32), and so a weight by dz, relative; weights are rounded to the
type of V where the products run on tensor cores (16-bit calls: the call's type, 4-bit cache: f16),
half a step e of it; the denominator sums the rounded weights, so with A = sum w |v| / sum w an
output moves by A (2 e + 2 dz).  f16 has a smallest step, 2^-24: the kernels hold the row's largest
weight at 2^5 and more, so a weight is off by 2^-30 of it, and N keys in one direction move an output
by 2^-30 w_max (sum |v| + N |out|) / sum w.  bf16 has no such step within 100 powers of two.  Each step of 16
keys rounds the running sum once, or cuts its addends, by 2^-23 of it at most: under (N / 16 + 16)
2^-22 A.  The output is rounded once."""
import pytest
import torch

from gqa_canvas_attention_gb300 import binding as B
from test_serving_gpu import E2M1, F64, TYPES, _lib, check_attention, gen, half_step, tiny  # noqa: F401

pytestmark = pytest.mark.gpu


def plain(q, k, v, scale, first, weight_type):
    """(values, tolerance) of query rows that see the keys from `first` (an index a row) on, in 64 bits."""
    nh, nkv, N = q.shape[2], k.shape[2], k.shape[1]
    want = torch.zeros(q.shape, dtype=F64, device="cuda")
    tol = torch.zeros_like(want)
    e = 0.0 if weight_type is None else half_step(weight_type)
    see = torch.arange(N, device="cuda")[None] >= first[:, None]
    for b in range(q.shape[0]):
        for h in range(nh):
            kk, vv, qq = k[b, :, h // (nh // nkv)].double(), v[b, :, h // (nh // nkv)].double(), q[b, :, h].double()
            hidden = ~see.any(0)
            kk[hidden], vv[hidden] = 0, 0
            z = (qq @ kk.T * scale).masked_fill(~see, -torch.inf)
            dz = (2.0 ** -21 * abs(scale) * (qq.abs() @ kk.abs().T)).masked_fill(~see, 0).amax(-1, keepdim=True)
            w = torch.softmax(z, -1)
            y, a = w @ vv, w @ vv.abs()
            t = y.abs() * half_step(q.dtype) * 1.01 + tiny(q.dtype) + a * (2 * e + 2 * dz + (N / 16 + 16) * 2.0 ** -22)
            if weight_type is torch.float16:
                t += 2.0 ** -30 * w.amax(-1, keepdim=True) * (see.double() @ vv.abs() + N * y.abs())
            want[b, :, h], tol[b, :, h] = y, t
    return want, tol


def sink_rows(T, nh, hd, dt, g):
    """Queries whose first element picks out a key's lead; the others spread the scores by about one."""
    q = torch.randn(1, T, nh, hd, generator=g, device="cuda") * (1.4 / hd ** 0.5)
    q[..., 0] = 1.0
    return q.to(dt)


LEADS = [13, 18, 20, 21, 24]              # log2 units


@pytest.mark.parametrize("dt", ["f16", "bf16"])
@pytest.mark.parametrize("hd", [64, 128, 256])
@pytest.mark.parametrize("T,N,at", [(1, 4096, 0), (1, 32768, 0), (4, 8192, 5000), (150, 4096, 0), (150, 8192, 8191),
                                    (700, 8192, 0), (300, 32768, 3)])
def test_a_key_that_leads(T, N, at, hd, dt):
    """Key `at` has value 0 and leads the others, whose values are about 1 and whose weights together matter."""
    nh, nkv = 2, 1
    g = gen(N + T + hd)
    q = sink_rows(T, nh, hd, TYPES[dt], g)
    plan = B.WindowPlan(nh, nkv, hd, 1, T, N)
    for lead in LEADS:
        k = torch.randn(1, N, nkv, hd, generator=g, device="cuda") * 0.5
        v = 1 + 0.25 * torch.randn(1, N, nkv, hd, generator=g, device="cuda")
        k[..., 0] = 0
        k[:, at] = 0
        k[:, at, :, 0] = lead * 0.6931472
        v[:, at] = 0
        k, v = k.to(TYPES[dt]), v.to(TYPES[dt])
        out = plan.attend(q, k, v)
        want, tol = plain(q, k, v, 1.0, torch.zeros(T, device="cuda"), TYPES[dt])
        check_attention(out, want, tol, f"lead {lead}")
    assert plan.sync_status() == B.DG_OK


@pytest.mark.parametrize("dt", ["f16", "bf16"])
@pytest.mark.parametrize("hd", [64, 128, 256])
@pytest.mark.parametrize("T,N,at", [(1, 32768, 0), (4, 8192, 5000), (150, 4096, 0), (700, 8192, 0), (300, 32768, 3)])
def test_a_key_that_leads_4_bit(T, N, at, hd, dt):
    nh, nkv = 2, 1
    g = gen(N + T + hd)
    q = sink_rows(T, nh, hd, TYPES[dt], g)
    plan = B.WindowPlan(nh, nkv, hd, 1, T, N)
    grid = torch.tensor(E2M1 + [-y for y in E2M1], dtype=F64, device="cuda")

    def values(code, scale):
        x = grid[torch.stack([code & 15, code >> 4], -1).flatten(-2).long()]
        return (x * scale.view(torch.float8_e4m3fn).double().repeat_interleave(16, -1)).transpose(1, 2)

    for lead in LEADS:
        # K of +-.5 (code 1 or 9, scale 1) and the lead in the key's first element: 3 x 16ths; V of 1 (code 2)
        # and 1.5 (code 3)
        cache = B.Kv4Cache(1, nkv, N, hd)
        bit = lambda n: torch.randint(0, 2, (1, nkv, N, n), generator=g, device="cuda", dtype=torch.uint8)
        cache.k.copy_((1 + 8 * bit(hd // 2)) | (1 + 8 * bit(hd // 2)) << 4)
        cache.v.copy_((2 + bit(hd // 2)) | (2 + bit(hd // 2)) << 4)
        cache.k_scale.fill_(0x38)
        cache.v_scale.fill_(0x38)
        cache.k[..., 0] &= 0xF0
        cache.k[:, :, at] = 0
        cache.v[:, :, at] = 0
        cache.k[:, :, at, 0] = 5                                             # 3
        byte = torch.tensor([lead * 0.6931472 / 3]).to(torch.float8_e4m3fn).view(torch.uint8)
        cache.k_scale[:, :, at] = int(byte)
        out = plan.attend_kv4(q, cache)
        want, tol = plain(q, values(cache.k, cache.k_scale), values(cache.v, cache.v_scale), 1.0,
                          torch.zeros(T, device="cuda"), torch.float16)
        check_attention(out, want, tol, f"lead {lead}")
    assert plan.sync_status() == B.DG_OK


@pytest.mark.parametrize("dt", ["f16", "bf16"])
@pytest.mark.parametrize("T,hd", [(3, 64), (150, 128), (150, 256)])
def test_a_key_that_leads_beside_a_hidden_nan(T, hd, dt):
    """Rows that are computed once more, since a NaN stands in a key that only the first row sees."""
    N, nh, nkv = 3000, 2, 1
    g = gen(T)
    q = sink_rows(T, nh, hd, TYPES[dt], g)
    k = torch.randn(1, N, nkv, hd, generator=g, device="cuda") * 0.5
    v = 1 + 0.25 * torch.randn(1, N, nkv, hd, generator=g, device="cuda")
    left = N - T - 1                                       # row t sees the keys from t + 1 on
    k[..., 0], k[:, T] = 0, 0
    k[:, T, :, 0], v[:, T] = 20 * 0.6931472, 0
    v[:, 1] = float("nan")
    k, v = k.to(TYPES[dt]), v.to(TYPES[dt])
    plan = B.WindowPlan(nh, nkv, hd, 1, T, N)
    out = plan.attend(q, k, v, left=left)
    assert torch.isnan(out[:, 0]).all()
    want, tol = plain(q[:, 1:], k, v, 1.0, torch.arange(2, T + 1, device="cuda"), TYPES[dt])
    check_attention(out[:, 1:], want, tol)
