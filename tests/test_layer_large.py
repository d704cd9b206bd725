"""Activations above the sizes from which rows are read past the caches: the bits of the
same rows in slices below them."""
import pytest
import torch

pytestmark = pytest.mark.gpu

import blockwise_fp8_gemm_bfp8_amd as bfp8  # noqa: E402
from layer_cases import generator, padded  # noqa: E402

BF = torch.bfloat16
GATE, NORM = 64 << 20, 32 << 20  # bytes of gate and of x, above which a call is a large one


def sliced(rows, step):
    return [slice(at, min(at + step, rows)) for at in range(0, rows, step)]


@pytest.mark.parametrize("cols", [4100, 4104, 4097])  # with tails and without
def test_gated_activation(cols):
    rows = GATE // (2 * cols) + 9
    assert rows * cols * 2 > GATE
    gen = generator(cols)
    gate, up = padded(rows, cols, BF, gen, 3.0), padded(rows, cols, BF, gen, 1.5, 1)
    dh = padded(rows, cols, BF, gen, 1e-3)
    h = bfp8.swiglu(gate, up)
    dgate, dup = bfp8.swiglu_backward(dh, gate, up)
    for at in sliced(rows, 3000):
        assert torch.equal(h[at], bfp8.swiglu(gate[at], up[at]))
        a, b = bfp8.swiglu_backward(dh[at], gate[at], up[at])
        assert torch.equal(dgate[at], a) and torch.equal(dup[at], b)
    if cols % 8:  # padding stays
        out = padded(rows, cols, BF, gen)
        bfp8.swiglu(gate, up, out=out)
        assert torch.equal(out, h) and torch.all(out._base[:, cols:] == 777)
    # over its own inputs, the results crossed
    bfp8.swiglu_backward(dh, gate, up, dgate=up, dup=gate)
    assert torch.equal(up, dgate) and torch.equal(gate, dup)


def test_gated_activation_over_the_halves_of_one_projection():
    rows, cols = 8200, 4104
    gate_up = torch.randn((rows, 2 * cols), device="cuda", generator=generator(1)).to(BF)
    gate, up = gate_up[:, :cols], gate_up[:, cols:]
    want = torch.cat([bfp8.swiglu(gate[at], up[at]) for at in sliced(rows, 4000)])
    kept = up.clone()
    bfp8.swiglu(gate, up, out=gate)
    assert torch.equal(gate, want) and torch.equal(up, kept)


@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("added", [False, True])
@pytest.mark.parametrize("cols", [40, 300, 1001, 2050, 3900, 8185, 16383])
def test_norm(cols, added, in_place):
    rows = NORM // (2 * cols) + 9
    gen = generator(cols)
    x = padded(rows, cols, BF, gen, 2.0)
    residual = padded(rows, cols, BF, gen, 1.0, 1) if added else None
    w = 1 + 0.1 * torch.randn(cols, device="cuda", generator=gen)
    want = [bfp8.rmsnorm(x[at], w, residual[at] if added else None) for at in sliced(rows, rows // 2 + 1)]
    y, r, rstd = (torch.cat(t) for t in zip(*want))
    if not in_place:
        got = bfp8.rmsnorm(x, w, residual)
    elif added:
        got = bfp8.rmsnorm(x, w, residual, out=x, sum_out=residual)
        assert got[0] is x and got[1] is residual
    else:
        got = bfp8.rmsnorm(x, w, out=x)
        assert got[0] is x
    assert torch.equal(got[0], y) and torch.equal(got[2], rstd)
    if added or not in_place:
        assert torch.equal(got[1], r)
    if cols % 8:
        assert not in_place or torch.all(x._base[:, cols:] == 777)


@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("added", [False, True])
@pytest.mark.parametrize("transposed", [False, True])
@pytest.mark.parametrize("scales", ["fp32", "mx128", "mx32"])
def test_codes_of_the_norm(scales, transposed, added, in_place):
    rows, cols, part = 8192, 2176, 4096
    assert rows * cols * 2 > NORM > part * cols * 2
    gen = generator(5)
    x, w = padded(rows, cols, BF, gen, 2.0, 1), 1 + 0.1 * torch.randn(cols, device="cuda", generator=gen)
    residual = padded(rows, cols, BF, gen, 1.0) if added else None
    call = lambda at, **k: bfp8.rmsnorm_quantize(x[at], w, residual[at] if added else None, scales=scales,
                                                 transposed=transposed, **k)
    want = [call(at) for at in sliced(rows, part)]
    got = call(slice(0, rows), **({"sum_out": residual} if added and in_place else {}))
    q, s, *rest = zip(*want)
    major = scales != "mx32"  # K-block major scales: rows along the second axis, tokens along the first
    assert torch.equal(got[0], torch.cat(q)) and torch.equal(got[1], torch.cat(s, 1 if major else 0))
    if transposed:
        qt, st, *rest = rest
        assert torch.equal(got[2], torch.cat(qt, 1)) and torch.equal(got[3], torch.cat(st, 0 if major else 1))
    r, rstd = rest
    assert torch.equal(got[-2], torch.cat(r)) and torch.equal(got[-1], torch.cat(rstd))


def test_gradient_of_the_norm_over_large_rows():
    """dx row by row; dw is a sum in another order: within its own roundings."""
    rows, cols = 8200, 2050
    gen = generator(6)
    r, dy, dsum = (padded(rows, cols, BF, gen, s, e) for s, e in ((2.0, 0), (1e-3, 1), (1e-3, 0)))
    w = 1 + 0.1 * torch.randn(cols, device="cuda", generator=gen)
    _, _, rstd = bfp8.rmsnorm(r, w)
    dx, dw = bfp8.rmsnorm_backward(dy, r, w, rstd, dsum)
    total = torch.zeros(cols, dtype=torch.float64, device="cuda")
    for at in sliced(rows, 2736):  # rstd's slices start 16-byte aligned
        a, b = bfp8.rmsnorm_backward(dy[at], r[at], w, rstd[at], dsum[at])
        assert torch.equal(dx[at], a)
        total += b.double()
    size = (dy.double() * r.double() * rstd.double()[:, None]).abs().sum(0)
    # a sum of 8200 terms in either order passes at most 100 additions a term
    assert torch.all((dw.double() - total).abs() <= 200 * 2.0 ** -24 * size)
