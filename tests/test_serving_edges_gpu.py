"""Calls of the serving operators that their declarations allow, at the edges of what they hold.

Plain forms and tolerances are those of test_serving_gpu."""
import pytest
import torch

from gqa_canvas_attention_gb300 import binding as B
from test_serving_gpu import _lib, gen  # noqa: F401

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
