"""Calls of the serving operators that their declarations allow, at the edges of what they hold.

Plain forms and tolerances are those of test_serving_gpu."""
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
