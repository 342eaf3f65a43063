"""Which layouts the serving operators take: rows that share bytes are refused, slices of one buffer that
share none are not.  Stand-in addresses on a machine without a GPU: a call that is not refused ends at the
missing device."""
import random

import pytest
import torch

from gqa_canvas_attention_gb300 import binding as B
from gqa_canvas_attention_gb300 import build as build_mod
from test_serving import kv4, rope_args

BASE = 1 << 40


@pytest.fixture(scope="module")
def lib():
    if torch.cuda.is_available():
        pytest.skip("stand-in addresses: for machines without a GPU")
    build_mod.build()
    return B.load()


def units(at, strides, sizes, hd, size):
    """The 16-byte units of a tensor's rows."""
    return {(at + (b * strides[0] + t * strides[1] + h * strides[2]) * size) // 16 + i
            for b in range(sizes[0]) for t in range(sizes[1]) for h in range(sizes[2]) for i in range(hd * size // 16)}


def layout(r, sizes, hd):
    """Strides of a padded buffer of these sizes with its dimensions in any order."""
    strides, step = [0, 0, 0], hd + 8 * r.choice([0, 0, 1, 8])
    for d in r.sample(range(3), 3):
        strides[d] = step
        step = step * sizes[d] + 8 * r.choice([0, 0, 0, 1, 8])
    return strides


def call(lib, rope, at, strides, out_at, out_strides, sizes, in_type=1, out_type=1):
    rows = {0: (at, *strides), 3: (out_at, *out_strides)}
    args = rope_args(batch=sizes[0], T=sizes[1], nh=sizes[2], nkv=0, hd=64, in_type=in_type, out_type=out_type,
                     rows={**rows, 1: (0,) * 4, 2: (0,) * 4, 4: (0,) * 4, 5: (0,) * 4}, positions=BASE >> 1)
    return lib.dg_attn_rope_apply(rope.handle, args, None)


def test_slices_of_one_buffer(lib):
    """q and its output as slices of one buffer, any order of dimensions, any distance."""
    r = random.Random(7)
    rope = B.Rope(64)
    taken = refused = 0
    for _ in range(3000):
        sizes = [r.randint(1, 4), r.randint(1, 5), r.randint(1, 4)]
        whole = [n + r.randint(0, 4) for n in sizes]
        strides = layout(r, whole, 64)
        offset = sum(s * r.randint(0, w - n) for s, w, n in zip(strides, whole, sizes))
        if r.random() < 0.2:
            offset += 8 * r.randint(-8, 8)
        at, out_at = BASE, BASE + 2 * offset
        if offset == 0:
            continue                                         # in place
        share = units(at, strides, sizes, 64, 2) & units(out_at, strides, sizes, 64, 2)
        rc = call(lib, rope, at, strides, out_at, strides, sizes)
        assert rc == (B.DG_ERR_ARG if share else B.DG_ERR_CUDA), (sizes, strides, offset, bool(share))
        taken, refused = taken + (not share), refused + bool(share)
    assert taken > 500 and refused > 300


def test_two_layouts(lib):
    """Input and output of strides and types of their own."""
    r = random.Random(8)
    rope = B.Rope(64)
    taken = refused = 0
    for _ in range(3000):
        sizes = [r.randint(1, 3), r.randint(1, 5), r.randint(1, 4)]
        in_type, out_type = r.choice([0, 1, 2]), r.choice([0, 1, 2])
        size = lambda t: 4 if t == 0 else 2
        a, b = layout(r, [n + r.randint(0, 3) for n in sizes], 64), layout(r, [n + r.randint(0, 3) for n in sizes], 64)
        if r.random() < 0.3:
            a = [0 if r.random() < 0.5 else x for x in a]    # an input may repeat
        out_at = BASE + 16 * r.randint(-700, 700)
        share = units(BASE, a, sizes, 64, size(in_type)) & units(out_at, b, sizes, 64, size(out_type))
        rc = call(lib, rope, BASE, a, out_at, b, sizes, in_type, out_type)
        assert rc == (B.DG_ERR_ARG if share else B.DG_ERR_CUDA), (sizes, a, b, out_at - BASE, in_type, out_type)
        taken, refused = taken + (not share), refused + bool(share)
    assert taken > 500 and refused > 500


def test_heads_outside_tokens_in_place(lib):
    """q, k and v of one [batch, heads, T, hd] buffer, rotated in place."""
    nh, nkv, T, hd = 4, 2, 7, 64
    H = nh + 2 * nkv
    rope = B.Rope(hd)
    rows = {}
    for i, first in enumerate((0, nh, nh + nkv)):
        rows[i] = rows[i + 3] = (BASE + 2 * first * T * hd, H * T * hd, hd, T * hd)
    args = rope_args(batch=3, T=T, nh=nh, nkv=nkv, hd=hd, rows=rows, positions=BASE >> 1)
    assert lib.dg_attn_qk_norm_rope(rope.handle, args, None) == B.DG_ERR_CUDA
    rows[4] = (BASE + 2 * (nh * T * hd - hd), H * T * hd, hd, T * hd)        # k's output over q's last row
    args = rope_args(batch=3, T=T, nh=nh, nkv=nkv, hd=hd, rows=rows, positions=BASE >> 1)
    assert lib.dg_attn_qk_norm_rope(rope.handle, args, None) == B.DG_ERR_ARG


def test_strides_beyond_the_address_space(lib):
    rope = B.Rope(64)
    for s in (1 << 62, -(1 << 63), 1 << 57):
        assert call(lib, rope, BASE, [s, 256, 64], BASE << 1, [768, 256, 64], [2, 3, 4]) == B.DG_ERR_ARG
        assert call(lib, rope, BASE, [768, 256, 64], BASE << 1, [s, 256, 64], [2, 3, 4]) == B.DG_ERR_ARG
    top = 2 ** 31 - 1
    assert lib.dg_attn_kv4_append(kv4(batch=top, nkv=top, cap=top), None, None) == B.DG_ERR_ARG


def test_outputs_of_absent_tensors():
    """An output for a tensor that is not there would come back as it was."""
    q, pos = torch.zeros(2, 3, 4, 64, dtype=torch.float16), torch.zeros(2, 3, dtype=torch.int64)
    build_mod.build()
    rope = B.Rope(64)
    with pytest.raises(ValueError, match="k_out without k"):
        rope.apply(q, None, pos, k_out=q)
    with pytest.raises(ValueError, match="k_out without k"):
        rope.qk_norm(q, None, None, pos, k_out=q)
    with pytest.raises(ValueError, match="v_out without v"):
        rope.qk_norm(q, q, None, pos, v_out=q)
