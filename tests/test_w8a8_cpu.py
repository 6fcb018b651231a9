"""Host-side checks of the int8 mode's 8-bit products that need no GPU: arguments are refused
before anything is launched, workspace sizes, shape checks of the wrappers."""
import pytest

from w4_gemm_amd import _lib
from w4_gemm_amd import shapes as S

BIG = 1 << 44


def _payload(n=16, k=256, rank=16, reserved=0, codes=0x1000, scales=0x2000, up=0x3000, down=0x4000):
    return _lib.SqW8(n, k, rank, reserved, codes, scales, up, down)


def _calls(p, m=4, a=0x8000, out=0x9000, dt=0, ws=0xA000, nb=BIG, offsets=0xB000, groups=2):
    return [_lib.sq_linear_fwd_w8a8(a, m, p, out, dt, ws, nb, None),
            _lib.sq_linear_dgrad_w8(a, m, p, out, dt, ws, nb, None),
            _lib.sq_grouped_fwd_w8a8(a, m, offsets, groups, p, out, dt, ws, nb, None),
            _lib.sq_grouped_dgrad_w8(a, m, offsets, groups, p, out, dt, ws, nb, None)]


BAD = [
    ("k not multiple of 256", dict(k=300), 2),
    ("k past the limit", dict(k=65536 + 256), 2),
    ("n < 1", dict(n=0), 2),
    ("n past 32 bits", dict(n=1 << 31), 2),
    ("rank 8", dict(rank=8), 4),
    ("reserved set", dict(reserved=1), 4),
    ("null codes", dict(codes=None), 1),
    ("null scales", dict(scales=None), 1),
    ("null up with rank", dict(up=None), 1),
    ("misaligned codes", dict(codes=0x1008), 5),
    ("misaligned down", dict(down=0x4002), 5),
]


@pytest.mark.parametrize("why,kw,status", BAD, ids=[b[0] for b in BAD])
def test_payload_is_refused(why, kw, status):
    assert _calls(_payload(**kw)) == [status] * 4


def test_arguments_are_refused():
    p = _payload()
    assert _calls(p, m=-1) == [2] * 4
    assert _calls(p, m=1 << 31) == [2] * 4
    assert _calls(p, dt=2) == [7] * 4
    assert _calls(p, a=None) == [1] * 4
    assert _calls(p, out=None) == [1] * 4
    assert _calls(p, ws=None) == [1] * 4
    assert _calls(p, a=0x8004) == [5] * 4
    assert _calls(p, out=0x9008) == [5] * 4
    assert _calls(p, ws=0xA001) == [5] * 4
    assert _calls(p, nb=0) == [6] * 4
    assert _calls(p, m=0, a=None, out=None, ws=None, nb=0, offsets=None) == [0] * 4   # no-op
    assert _calls(p, offsets=None)[2:] == [1, 1]
    assert _calls(p, offsets=0xB004)[2:] == [5, 5]
    assert _calls(p, groups=0)[2:] == [2, 2]
    assert _calls(p, groups=-3)[2:] == [2, 2]
    assert _calls(p, m=1 << 30, groups=1 << 20)[2:] == [2, 2]
    # the gradient's sums are exact up to N = 131072 only
    big = _payload(n=131073)
    assert _lib.sq_linear_dgrad_w8(0x8000, 4, big, 0x9000, 0, 0xA000, BIG, None) == 2
    assert _lib.sq_linear_dgrad_w8_workspace_bytes(4, big) == 0
    assert _lib.sq_linear_fwd_w8a8_workspace_bytes(4, big) > 0


def test_workspace_bytes():
    for rank in (0, 16, 32, 64):
        p = _payload(n=100, k=512, rank=rank)
        last = 0
        for m in (1, 16, 17, 300, 5000):
            f, d = _lib.sq_linear_fwd_w8a8_workspace_bytes(m, p), _lib.sq_linear_dgrad_w8_workspace_bytes(m, p)
            assert f >= m * 512 + 4 * m + 4 * m * rank        # integers, scales, one slice of t
            assert d >= 2 * m * 128 + 4 * m + 4 * m * rank    # rows padded to 64
            assert _lib.sq_grouped_fwd_w8a8_workspace_bytes(m, 1, p) == f
            assert _lib.sq_grouped_dgrad_w8_workspace_bytes(m, 1, p) == d
            assert f > last
            last = f
            for fn, grouped, nb in ((_lib.sq_linear_fwd_w8a8, _lib.sq_grouped_fwd_w8a8, f),
                                    (_lib.sq_linear_dgrad_w8, _lib.sq_grouped_dgrad_w8, d)):
                assert fn(0x8000, m, p, 0x9000, 0, 0xA000, nb - 1, None) == 6
                assert grouped(0x8000, m, 0xB000, 1, p, 0x9000, 0, 0xA000, nb - 1, None) == 6
    p = _payload()
    for m, groups in ((0, 1), (-1, 1), (4, 0), (1 << 31, 1)):
        assert _lib.sq_grouped_fwd_w8a8_workspace_bytes(m, groups, p) == 0
        assert _lib.sq_grouped_dgrad_w8_workspace_bytes(m, groups, p) == 0
    assert _lib.sq_linear_fwd_w8a8_workspace_bytes(4, _payload(rank=24)) == 0


def test_gradient_of_too_many_rows_is_refused():
    """A gradient launch has fewer than 2^32 threads: 2^25 rows, 2^23 of more than 2048 values."""
    for n, most in ((1, 1 << 25), (2048, 1 << 25), (2049, 1 << 23)):
        p = _payload(n=n, k=256)
        assert _lib.sq_linear_dgrad_w8_workspace_bytes(most, p) > 0
        assert _lib.sq_linear_dgrad_w8_workspace_bytes(most + 1, p) == 0
        assert _lib.sq_grouped_dgrad_w8_workspace_bytes(most + 1, 2, p) == 0
        assert _lib.sq_linear_dgrad_w8(0x8000, most + 1, p, 0x9000, 0, 0xA000, 1 << 60, None) == 2
        assert _lib.sq_linear_fwd_w8a8_workspace_bytes(most + 1, p) > 0


def test_status_text_names_the_limits():
    assert "65536" in _lib.status_str(2) and "131072" in _lib.status_str(2)


def test_grouped_payload_shapes():
    ok = ((3, 8, 512), (3, 8), (3, 8, 16), (3, 512, 16))
    assert S.check_grouped_w8_payload(*ok) == (3, 8, 512, 16)
    assert S.check_grouped_w8_payload((1, 5, 256), (1, 5), None, None) == (1, 5, 256, 0)
    bad = [
        ((8, 512), (8,), None, None),                              # not stacked
        ((0, 8, 512), (0, 8), None, None),                         # no experts
        ((3, 8, 500), (3, 8), None, None),                         # K
        ((3, 8, 512), (3, 9), None, None),                         # scales
        ((3, 8, 512), (3, 8), (8, 16), (512, 16)),                 # factors not stacked
        ((3, 8, 512), (3, 8), (2, 8, 16), (2, 512, 16)),           # factors of fewer experts
        ((3, 8, 512), (3, 8), (3, 8, 16), None),                   # one factor missing
        ((3, 8, 512), (3, 8), (3, 8, 8), (3, 512, 8)),             # rank 8
    ]
    for args in bad:
        with pytest.raises(ValueError):
            S.check_grouped_w8_payload(*args)
    S.check_offsets((4,), 3)
    for shp in ((3,), (5,), (4, 1), ()):
        with pytest.raises(ValueError):
            S.check_offsets(shp, 3)
