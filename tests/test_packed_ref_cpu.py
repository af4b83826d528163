"""The 64-bit values that the packed and paged tests compare with (tests/packed_ref.py), head by
head and sequence by sequence against the oracle; and mistakes planted in copies of them, which
the oracle tells from the values and the tests' bounds tell from the kernels' roundings."""
import numpy as np
import pytest
import torch

import oracle
from tests import packed_ref

NAMES = ("O", "L", "dQ", "dK", "dV")


@pytest.fixture(scope="module")
def orc():
    oracle.build()
    return oracle.Oracle(oracle.LIBRARY)


def _case(causal):
    lens, hq, hkv, d, scale = [5, 0, 33, 1, 70], 6, 2, 16, 0.21
    q, k, v, do, _ = packed_ref.packed_inputs(lens, hq, hkv, d, 3, rest=2, device="cpu")
    return q, k, v, lens, causal, scale, do


def _oracle(orc, q, k, v, lens, causal, scale, do):
    """The packed layout from the oracle's single heads: O, dQ, L, dK, dV (rows of sequences)."""
    x = [t.double().numpy() for t in (q, k, v, do)]
    n, hq, hkv = sum(lens), q.shape[1], k.shape[1]
    out = {"O": np.zeros((n, hq, q.shape[2])), "L": np.zeros((hq, n))}
    out["dQ"], out["dK"], out["dV"] = np.zeros_like(out["O"]), *(
        np.zeros((n, hkv, q.shape[2])) for _ in range(2))
    at = 0
    for m in lens:
        r = slice(at, at + m)
        at += m
        for h in range(hq if m else 0):
            hk = h // (hq // hkv)
            part = [x[0][r, h], x[1][r, hk], x[2][r, hk], x[3][r, h]]
            out["O"][r, h], out["L"][h, r] = orc.forward(*part[:3], causal, scale)
            dq, dk, dv, _ = orc.backward(*part, causal, scale)
            out["dQ"][r, h] = dq
            out["dK"][r, hk] += dk
            out["dV"][r, hk] += dv
    return {name: torch.from_numpy(t) for name, t in out.items()}


def _rows(name, t, n):
    return t[:, :n] if name == "L" else t[:n]


def _differs(got, want, n):
    return [name for name in NAMES
            if not torch.allclose(_rows(name, got[name][0], n), want[name], rtol=1e-10, atol=1e-12)]


@pytest.mark.parametrize("causal", [True, False])
def test_values_are_the_oracles(orc, causal):
    case = _case(causal)
    got = packed_ref.packed64(*case)
    n = sum(case[3])
    assert _differs(got, _oracle(orc, *case), n) == []
    for name in NAMES:
        value, bound = (_rows(name, x, n) for x in got[name])
        assert torch.isfinite(value).all() and (bound >= 0).all()
    assert torch.isnan(got["O"][0][n:]).all()  # rows of no sequence have no value


MISTAKES = {
    "mask_off_by_one": (".triu(1)", ".triu(2)"),
    "dS_sign": ("ds = p * (dp - D)", "ds = p * (dp + D)"),
    "dQ_drops_scale": ("dq = scale * torch.matmul(ds, k)", "dq = torch.matmul(ds, k)"),
    "dK_drops_scale": ("dk = scale * torch.matmul(", "dk = torch.matmul("),
    "one_head_too_far": ("hs = slice(h * g, (h + 1) * g)", "hs = slice(h, hq, hkv)"),
    "gradients_of_one_head": ("dv = torch.matmul(pt, do).sum(0)", "dv = torch.matmul(pt, do)[0]"),
    "sequences_run_on": ("rows = slice(at, at + n)", "rows = slice(max(0, at - 1), at + n)"),
    "L_of_base_two": ("L = torch.logsumexp(s, dim=-1)",
                      "L = torch.logsumexp(s, dim=-1) / math.log(2)"),
}


@pytest.mark.parametrize("name", sorted(MISTAKES))
def test_planted_mistakes_are_caught(orc, name):
    before, after = MISTAKES[name]
    text = open(packed_ref.__file__).read()
    assert text.count(before) >= 1, f"no place for {name}"
    copy = {"__name__": "copy"}
    exec(compile(text.replace(before, after), f"packed_ref_{name}", "exec"), copy)
    case = _case(True)
    n = sum(case[3])
    got, right = copy["packed64"](*case), packed_ref.packed64(*case)
    assert _differs(got, _oracle(orc, *case), n) != []
    caught = []
    for out in NAMES:
        try:
            packed_ref.assert_close(out, _rows(out, got[out][0], n),
                                    tuple(_rows(out, x, n) for x in right[out]))
        except AssertionError:
            caught.append(out)
    assert caught, f"{name} is within the bounds of every output"
