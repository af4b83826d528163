"""The bounds of tests/cache4_ref.py: mistakes that O alone has to show, and the arithmetic that
they allow."""
import math

import pytest
import torch

from tests import cache4_ref, rope_ref as ref


def _case(n, d, g=4, seed=1):
    """Queries [g, d], codes and pairs of n keys for which every part of them counts."""
    gen = torch.Generator().manual_seed(seed + n + d)
    codes = torch.randint(0, 16, (2, 1, 1, n, d), generator=gen)
    scale = 0.05 + 0.3 * torch.rand(2, 1, 1, n, ref.groups(d), generator=gen)
    pairs = torch.stack([scale, -7.5 * scale], -1).to(torch.bfloat16).double()
    place = [(torch.zeros(n, dtype=torch.long), torch.arange(n))]
    q, pairs = cache4_ref.telling(torch.zeros(1, g, d), codes, pairs, place, seed)
    return q[0].double(), codes[:, 0, 0], pairs[:, 0, 0]


def _weights(q, codes, pairs, scale):
    return torch.softmax(cache4_ref.scores64(q, codes[0], pairs[0], scale), -1)


@pytest.mark.parametrize("n,parts,d", [(5000, 57, 128), (9000, 100, 40), (40000, 228, 128)])
def test_mistakes_that_the_bound_of_O_shows(n, parts, d):
    q, codes, pairs = _case(n, d)
    scale = 1 / math.sqrt(d)
    (o, bound), _ = cache4_ref.decode_bounds(q, codes, pairs, scale)
    p, v = _weights(q, codes, pairs, scale), ref.values(codes[1], pairs[1])
    one = n // parts  # keys of one part
    lost, swapped, twice = p.clone(), v.clone(), p.clone()
    lost[:, 7 * one:8 * one] = 0
    twice[:, 7 * one:8 * one] *= 2
    swapped[:one], swapped[7 * one:8 * one] = v[7 * one:8 * one], v[:one]
    for name, wrong, share in (
            ("nothing", torch.zeros_like(o), 0.3), ("a lost part", lost @ v, 0.3),
            ("a part twice", twice / twice.sum(-1, keepdim=True) @ v, 0.3),
            ("two parts' values exchanged", p @ swapped, 0.3),
            ("the same weights for all", v.mean(0).expand_as(o), 0.3),
            ("values of 16 rows before", p @ v.roll(16, 0), 0.3)):
        seen = ((wrong - o).abs() > bound).double().mean()
        assert seen > share, (name, float(seen))


@pytest.mark.parametrize("n", [2, 5, 20])
def test_weights_of_fewer_bits_are_seen(n):
    """fp16 weights are within the bound, bf16 ones are not."""
    q, codes, pairs = _case(n, 128, g=16)
    pairs[1, ..., 1] = -7.5 * pairs[1, ..., 0]  # values around 0
    pairs = pairs.to(torch.bfloat16).double()
    scale = 1 / math.sqrt(128)
    (o, bound), _ = cache4_ref.decode_bounds(q, codes, pairs, scale)
    p = _weights(q, codes, pairs, scale)
    s, m = cache4_ref.wide(pairs[1], 128)
    off = {}
    for t in (torch.float16, torch.bfloat16):
        ps = torch.stack([(p * s[:, c]).to(t).double() @ codes[1][:, c].double()
                          for c in range(128)], -1)
        got = (ps + p @ m).to(torch.bfloat16).double()
        off[t] = ((got - o).abs() > bound).double().mean()
    assert off[torch.float16] == 0 and off[torch.bfloat16] > 0.001, off


def test_the_other_definition_agrees():
    q, codes, pairs = _case(300, 72)
    (o, _), (L, _) = cache4_ref.decode_bounds(q, codes, pairs, 0.1)
    (o2, _), (L2, _) = ref.decode64(q, codes, pairs, 0.1)
    assert torch.allclose(o, o2, rtol=1e-12, atol=1e-12) and torch.allclose(L, L2, rtol=1e-12)
