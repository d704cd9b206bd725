"""One token of tensors stored head by head with room for many: the strides of
an axis with one entry do not matter, however large the head's stride is."""
import numpy as np
import pytest
import torch

from oracle import attention as ref
from test_attention import f64, within

pytestmark = pytest.mark.gpu

import blockwise_fp8_gemm_bfp8_amd as bfp8  # noqa: E402

H, KV, D, ROOM = 16, 8, 128, 8192  # heads of 8192 rows of 128: a head's stride is 2^20


def one_token(heads, gen, at=0):
    room = torch.full((heads, ROOM, D), 7.0, dtype=torch.bfloat16, device="cuda")
    t = room[:, at:at + 1].transpose(0, 1)
    t.copy_(torch.randn((1, heads, D), device="cuda", generator=gen))
    return t, room


def alone(room, at):
    """The rows beside the token's are as they were."""
    return (room[:, :at] == 7).all() and (room[:, at + 1:] == 7).all()


@pytest.mark.parametrize("at", [0, 5000])
def test_rope(at):
    gen = torch.Generator(device="cuda").manual_seed(31)
    x, room = one_token(H, gen, at)
    table = bfp8.rope_table(ROOM, D)
    pos = torch.tensor([at], dtype=torch.int32, device="cuda")
    want = bfp8.rope(x.contiguous(), table, pos)
    assert torch.equal(bfp8.rope(x, table, pos), want)
    out, other = one_token(H, gen, at)
    bfp8.rope(x.contiguous(), table, pos, out=out)  # a rotated key into the cache
    assert torch.equal(out, want) and alone(other, at)
    bfp8.rope(x, table, pos, out=x)
    assert torch.equal(x, want) and alone(room, at)


@pytest.mark.parametrize("at", [0, 5000])
def test_attention_and_gradient(at):
    gen = torch.Generator(device="cuda").manual_seed(32)
    (q, _), (k, _), (v, _), (do, _) = (one_token(h, gen, at) for h in (H, KV, KV, H))
    (o, o_room), (dq, q_room), (dk, k_room), (dv, v_room) = (
        one_token(h, gen, at) for h in (H, H, KV, KV))
    _, lse = bfp8.attention_forward(q, k, v, out=o)
    args = ([0, 1], [0, 1], None, True, D ** -0.5)
    want, wl, ob, lb = ref.attention(f64(q), f64(k), f64(v), *args)
    within(o, want, ob, "o")
    within(lse, wl, lb, "lse")
    bfp8.attention_backward(do, q, k, v, o, lse, dq=dq, dk=dk, dv=dv)
    grads = ref.attention_gradient(f64(do), f64(q), f64(k), f64(v), *args)
    for i, t in enumerate((dq, dk, dv)):
        within(t, grads[i], grads[3 + i], "dq dk dv".split()[i])
    assert all(alone(room, at) for room in (o_room, q_room, k_room, v_room))


def test_first_step_over_a_cache():
    """The first generation step: a cache of one used row, sliced to it."""
    gen = torch.Generator(device="cuda").manual_seed(33)
    q = torch.randn((1, H, D), device="cuda", generator=gen).to(torch.bfloat16)
    (k, _), (v, _) = (one_token(KV, gen) for _ in range(2))
    o, lse = bfp8.attention_forward(q, k, v)
    want = v.repeat_interleave(H // KV, 1)  # one visible key: its value
    assert torch.equal(o, want) and np.isfinite(f64(lse)).all()
