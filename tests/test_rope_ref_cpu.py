"""The 64-bit values that the norm, rotation and 4-bit cache tests compare with: gradients
against differences, angles against complex numbers, the layout against its own rules."""
import pytest
import torch

import exact_io_aware_27_gb300 as fa
from tests import rope_ref as ref


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("d,rot", [(16, 16), (24, 8), (40, 40)])
def test_gradients_against_differences(d, rot, interleaved):
    g = torch.Generator().manual_seed(d + rot)
    x = torch.randn(3, 2, d, generator=g, dtype=torch.float64)
    w = torch.randn(d, generator=g, dtype=torch.float64)
    dy = torch.randn(3, 2, d, generator=g, dtype=torch.float64)
    cs, pos = fa.rope_table(50, rot, device="cpu"), torch.tensor([0, 49, 7])
    f = lambda x, w: (ref.norm_rope64(x, w, cs, pos, 1e-6, interleaved)[0] * dy).sum()  # noqa: E731
    dx, _, dw, _ = ref.norm_rope_backward64(dy, x, w, cs, pos, 1e-6, interleaved)
    h = 1e-6
    for t, grad, at in ((x, dx, 0), (w, dw, 1)):
        flat = t.view(-1)
        for i in range(flat.numel()):
            old = flat[i].item()
            flat[i] = old + h
            up = f(x, w)
            flat[i] = old - h
            down = f(x, w)
            flat[i] = old
            # differences: h^2 of the third derivative, and 2^-52 |f| / h of rounding
            assert abs((up - down) / (2 * h) - grad.view(-1)[i]) < 1e-7, (at, i)


def test_rotation_against_complex_numbers():
    cs = fa.rope_table(100000, 32, device="cpu")
    pos = torch.tensor([0, 1, 99999])
    x = torch.randn(3, 1, 40, dtype=torch.float64)
    c, s = ref.table64(cs, pos)
    for inter in (False, True):
        y, _ = ref.turn(x, c, s, inter)
        a, b = (x[..., 0:32:2], x[..., 1:32:2]) if inter else (x[..., :16], x[..., 16:32])
        z = torch.complex(a, b) * torch.complex(c, s)[:, None]
        got = (y[..., 0:32:2], y[..., 1:32:2]) if inter else (y[..., :16], y[..., 16:32])
        assert torch.allclose(got[0], z.real) and torch.allclose(got[1], z.imag)
        assert torch.equal(y[..., 32:], x[..., 32:])
        back, _ = ref.turn(y, c, s, inter, back=True)
        assert torch.allclose(back, x, atol=1e-6)  # the table's cos^2 + sin^2 is 1 to 2^-23


def test_table():
    t = fa.rope_table(70001, 64, base=500000.0, device="cpu").double()
    import math
    for p in (0, 1, 70000):
        for i in (0, 5, 31):
            a = p * 500000.0 ** (-2 * i / 64)
            assert abs(t[p, i] - math.cos(a)) < 2 ** -24 and abs(t[p, 32 + i] - math.sin(a)) < 2 ** -24
    for bad in ((0, 8), (8, 0), (8, 12)):
        with pytest.raises(ValueError):
            fa.rope_table(*bad, device="cpu")


@pytest.mark.parametrize("d", [64, 128])
def test_layout_covers_a_block_once(d):
    code, shift, pair = ref.places(d)
    nibbles = (2 * code + shift // 4).flatten().tolist()
    bytes_of_pairs = [b + i for b in pair.flatten().tolist() for i in range(4)]
    used = nibbles + [2 * b + i for b in bytes_of_pairs for i in (0, 1)]
    assert sorted(used) == list(range(2 * 1152 * ref.groups(d)))


@pytest.mark.parametrize("d", [8, 72, 128])
def test_pack_and_unpack(d):
    g = torch.Generator().manual_seed(d)
    like = torch.randint(0, 256, (3, 2, 2, 1152 * ref.groups(d)), generator=g).to(torch.uint8)
    codes = torch.randint(0, 16, (2, 3, 2, 32, d), generator=g)
    pairs = torch.randn(2, 3, 2, 32, ref.groups(d), 2, generator=g).to(torch.bfloat16).double()
    c, p = ref.unpack(ref.pack(codes, pairs, d, like), d)
    assert torch.equal(c, codes) and torch.equal(p, pairs)


def test_quantize_is_near():
    g = torch.Generator().manual_seed(1)
    for std, mean in ((1.0, 0.0), (1e-3, 100.0), (0.0, -3.1), (1e30, 0.0)):
        x = (torch.randn(50, 96, generator=g) * std + mean)
        codes, pairs = ref.quantize(x)
        scale, lo = (pairs.repeat_interleave(64, dim=-2)[..., :96, i] for i in (0, 1))
        off = (ref.values(codes, pairs) - x.double()).abs()
        assert (off <= torch.maximum(scale * (0.5 + 15 * ref.U), 2 * ref.U * lo.abs())).all()


def test_planted_mistakes_are_seen():
    """What the bounds have to tell apart."""
    g = torch.Generator().manual_seed(2)
    x = torch.randn(4, 2, 64, generator=g).to(torch.bfloat16)
    w = torch.randn(64, generator=g).to(torch.bfloat16)
    cs, pos = fa.rope_table(50, 64, device="cpu"), torch.tensor([3, 9, 20, 49])
    y, e = ref.norm_rope64(x, w, cs, pos, 1e-6, False)
    bound = ref.rounded(y, e)
    for wrong in (ref.norm_rope64(x, w, cs, pos + 0, 1e-6, True)[0],
                  ref.norm_rope64(x, w, cs, pos.clamp(max=48), 1e-6, False)[0],
                  ref.norm_rope64(x, None, cs, pos, 1e-6, False)[0],
                  ref.turn(ref.norm_rope64(x, w, None, pos, 1e-6, False)[0],
                           *ref.table64(cs, pos), False, back=True)[0]):
        assert ((wrong - y).abs() > bound).any()
    dy = torch.randn(4, 2, 64, generator=g).to(torch.bfloat16)
    dx, b, dw, bw = ref.norm_rope_backward64(dy, x, w, cs, pos, 1e-6, False)
    xx = x.double()
    r = 1 / torch.sqrt((xx * xx).mean(-1, keepdim=True) + 1e-6)
    gg = ref.turn(dy.double(), *ref.table64(cs, pos), False, back=True)[0]
    assert ((r * gg * w.double() - dx).abs() > b).any()       # without the mean's term
    assert (((gg * xx).sum((0, 1)) - dw).abs() > bw).any()    # without the norm
    q = torch.randn(3, 64, generator=g).to(torch.bfloat16).double()
    codes, pairs = ref.quantize(torch.randn(2, 40, 64, generator=g))
    (o, ob), (L, lb) = ref.decode64(q, codes, pairs, 0.125)
    for c, p in ((codes[:, :39], pairs[:, :39]), (codes.flip(0), pairs.flip(0)),
                 (codes, pairs * torch.tensor([1.0, 0.99])), (codes.clamp(max=14), pairs)):
        (o2, _), (L2, _) = ref.decode64(q, c, p, 0.125)
        assert ((o2 - o).abs() > ob).any() or ((L2 - L).abs() > lb).any()
