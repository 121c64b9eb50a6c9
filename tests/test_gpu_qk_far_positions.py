"""Angles of the norms with rotation at far positions, absolutely, against wide integers: rows with
one feature set, 8, have norm 8 and come back as 8 cos and 8 sin of one pair's angle.

Tolerance: as for every row, 16 roundings of half an fp32 step of the pair's norm and an angle
within 2^-24 pi (the fraction of a turn itself is good to 2^-31)."""
import numpy as np
import pytest

from tests.wide_turns import angle

torch = pytest.importorskip("torch")

pytestmark = pytest.mark.gpu
E = 2.0 ** -24
TOL = 8 * (16 * E + np.pi * 2.0 ** -24)
FAR = [0, 1, -1, 4095, 1 << 20, -(1 << 31), (1 << 31) + 5, (1 << 36) - 3, (1 << 40) + 12345, -(1 << 40) - 7, 3 ** 30, 1 << 52,
       -(1 << 52) + 11, (1 << 60) + 1, (1 << 62) + 987654321, (1 << 63) - 1, -(1 << 63)]
KINDS = [(64, False, 10000.0), (64, True, 10000.0), (48, False, 500000.0), (32, True, 1.0), (16, False, 1e6), (64, False, 3.7),
         (48, True, 1e300), (64, False, float(np.nextafter(1.0, 2.0)))]


@pytest.fixture(scope="module")
def dl():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from sparse_long_sequence_gb300 import binding
    return binding


def places(rot, interleaved, i):
    return (2 * i, 2 * i + 1) if interleaved else (i, i + rot // 2)


def unit_rows(rot, interleaved, n, which):
    """[1][rot / 2][n][64]: head i holds 8 in feature a (0) or b (1) of pair i."""
    x = torch.zeros(1, rot // 2, n, 64)
    for i in range(rot // 2):
        x[0, i, :, places(rot, interleaved, i)[which]] = 8
    return x.cuda()


def expected(rot, interleaved, theta, at):
    c, s = (np.array([[f(angle(p, theta, rot, i)) for p in at] for i in range(rot // 2)]) for f in (np.cos, np.sin))
    a, b = (np.zeros((1, rot // 2, len(at), 64)) for _ in range(2))
    for i in range(rot // 2):
        fa, fb = places(rot, interleaved, i)
        a[0, i, :, fa], a[0, i, :, fb] = 8 * c[i], 8 * s[i]
        b[0, i, :, fa], b[0, i, :, fb] = -8 * s[i], 8 * c[i]
    return a, b


@pytest.mark.parametrize("how", KINDS, ids=str)
@pytest.mark.parametrize("offset", [0, -(1 << 40) - 3], ids=["positions", "offset"])
def test_angles(dl, how, offset):
    rot, inter, theta = how
    # what the call adds up stays an int64
    at = [p for p in FAR if -(1 << 63) <= p - offset < 1 << 63]
    pos = torch.tensor([[p - offset for p in at]], dtype=torch.int64, device="cuda")
    q, k = unit_rows(rot, inter, len(at), 0), unit_rows(rot, inter, len(at), 1)
    got = dl.diffuser_qk_norm_rope(q, k, positions=pos, position_offset=offset, eps=1e-30, theta=theta, rotary_dim=rot,
                                   interleaved=inter)
    for g, ref in zip(got, expected(rot, inter, theta, at)):
        err = np.abs(g.double().cpu().numpy() - ref).max(axis=(0, 1, 3))
        assert (err <= TOL).all(), dict(zip(at, err))


@pytest.mark.parametrize("how", KINDS, ids=str)
def test_angles_backward(dl, how):
    # inputs with all their norm in a feature of another pair: dx = R(-p) dy
    rot, inter, theta = how
    pos = torch.tensor([FAR], dtype=torch.int64, device="cuda")
    q, k = unit_rows(rot, inter, len(FAR), 0).roll(1, 1).contiguous(), unit_rows(rot, inter, len(FAR), 1).roll(1, 1).contiguous()
    dy = unit_rows(rot, inter, len(FAR), 0), unit_rows(rot, inter, len(FAR), 1)
    got = dl.diffuser_qk_norm_rope_backward(q, k, *dy, positions=pos, eps=1e-30, theta=theta, rotary_dim=rot,
                                            interleaved=inter)[:2]
    back = expected(rot, inter, theta, [-p for p in FAR])
    for g, ref in zip(got, back):
        err = np.abs(g.double().cpu().numpy() - ref).max(axis=(0, 1, 3))
        assert (err <= 2 * TOL).all(), dict(zip(FAR, err))


def test_offset_alone(dl):
    # a single new token far out, without positions
    for p in ((1 << 52) + 3, -(1 << 60)):
        q, k = unit_rows(64, False, 1, 0), unit_rows(64, False, 1, 1)
        got = dl.diffuser_qk_norm_rope(q, k, position_offset=p, eps=1e-30)
        for g, ref in zip(got, expected(64, False, 10000.0, [p])):
            assert np.abs(g.double().cpu().numpy() - ref).max() <= TOL


def test_digits_near_quarter_turns(dl):
    # sines near half turns and cosines near odd quarter turns are small: they keep their digits.
    # Within 2^-31 turns and eight fp32 steps of the value: the angle's own rounding, the sine's, the
    # norm's and three products'.
    p = np.arange(1, 1 << 21)
    part = p / (2 * np.pi) % 0.25
    at = [int(x) for x in p[np.minimum(part, 0.25 - part) < 2.0 ** -13]][:800]
    assert 355 in at and 11 not in at and len(at) > 300
    q, k = unit_rows(16, False, len(at), 0), unit_rows(16, False, len(at), 1)
    pos = torch.tensor([at], dtype=torch.int64, device="cuda")
    for sign in (1, -1):
        got = dl.diffuser_qk_norm_rope(q, k, positions=sign * pos, eps=1e-30, theta=1.0, rotary_dim=16)
        for g, ref in zip(got, expected(16, False, 1.0, [sign * a for a in at])):
            err = np.abs(g.double().cpu().numpy() - ref) - 8 * 2 * np.pi * 2.0 ** -31 - 8 * E * np.abs(ref)
            assert err.max() <= 0, err.max()
