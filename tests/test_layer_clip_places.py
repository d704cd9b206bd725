"""Clipping refuses gradients whose memory would be written twice or while another job
reads it, wherever the overlap begins; what merely lies between one another is taken."""
import itertools
import random

import pytest
import torch

import blockwise_fp8_gemm_bfp8_amd as bfp8
from blockwise_fp8_gemm_bfp8_amd.layer import _meet, _refuse_overlaps, _span
from layer_cases import f64, generator
from oracle import layer


def bytes_of(span):
    at, rows, width, ld = span
    return {at + i * ld + k for i in range(rows) for k in range(width)}


def test_places_that_meet():
    """Against the sets of their bytes."""
    rng = random.Random(0)
    found = [0, 0]
    for _ in range(4000):
        a, b = (_span(rng.randrange(60), rows := rng.randint(1, 5), cols := rng.randint(1, 6),
                      cols + rng.choice([0, 0, 1, 5, 9]), rng.choice([2, 4])) for _ in range(2))
        meet = bool(bytes_of(a) & bytes_of(b))
        assert _meet(a, b) == _meet(b, a) == meet, (a, b)
        found[meet] += 1
    assert min(found) > 500


def test_lists_of_places():
    """Every pair is looked at, and pairs that are only read are not."""
    rng = random.Random(1)
    found = [0, 0]
    for _ in range(3000):
        places = [(rng.randrange(400), rng.randint(1, 4), rng.randint(1, 9), rng.randint(9, 20), 2, i,
                   rng.choice(["out", "grads"])) for i in range(5)]
        bad = any(bytes_of(_span(*a)) & bytes_of(_span(*b)) and "out" in (a[6], b[6])
                  for a, b in itertools.combinations(places, 2))
        try:
            _refuse_overlaps(places)
            refused = False
        except ValueError:
            refused = True
        assert refused == bad, places
        found[bad] += 1
    assert min(found) > 300


@pytest.mark.gpu
def test_refusals():
    buf, other = torch.ones(4000, device="cuda"), torch.ones(4000, device="cuda")
    rows = torch.ones((40, 100), device="cuda")
    half = torch.ones(4000, dtype=torch.bfloat16, device="cuda")
    for grads, out in (([buf[:1000], buf[500:1500]], None),           # shifted
                       ([buf, buf[3999:]], None),                     # the last element
                       ([buf[1000:], buf[:3000]], None),
                       ([buf[:1000]], [buf[4:1004]]),                 # onto itself, shifted
                       ([buf[:1000], buf[2000:3000]], [other[:1000], buf[900:1900]]),  # another's gradient
                       ([buf[:1000], buf[2000:3000]], [other[:1000], other[999:1999]]),
                       ([rows[:, :60], rows[:, 59:]], None),          # one column of two
                       ([rows[:, :10], rows.view(-1)[4:6]], None),    # a piece inside a row
                       ([half.view(torch.float32), half[10:20]], None)):
        with pytest.raises(ValueError, match="share memory"):
            bfp8.GradClip(grads, out)
        with pytest.raises(ValueError, match="share memory"):
            bfp8.clip_grads(grads, 1.0, out)


@pytest.mark.gpu
def test_neighbours_are_taken():
    """Views of one buffer that share nothing, in place."""
    base = torch.randn((64, 96), device="cuda", generator=generator(1))
    flat = torch.randn(1000, device="cuda", generator=generator(2))
    grads = [base[:, :32], base[:, 64:], base[:, 32:64], flat[:333], flat[333:], flat[5:5]]
    before = [f64(g) for g in grads]
    norm = bfp8.clip_grads(grads, 1.0)
    want = layer.grad_norm(before)
    assert abs(norm.item() - want) <= 2.0 ** -23 * want
    for g, b in zip(grads, before):
        assert abs(f64(g) - b / want).max(initial=0) <= 2.0 ** -21 * abs(b / want).max(initial=0)
    # gradients that are read only may be one another's: each counts
    twice = bfp8.grad_norm([flat, flat, flat[10:20]])
    want = layer.grad_norm([f64(t) for t in (flat, flat, flat[10:20])])
    assert abs(twice.item() - want) <= 2.0 ** -23 * want
    a, b = torch.empty_like(flat), torch.empty_like(flat)
    bfp8.clip_grads([flat, flat], 0.5, [a, b])
    assert torch.equal(a, b)
