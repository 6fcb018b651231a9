"""Host-side checks of the 8-bit float mode that need no GPU: arguments are refused before anything
is launched, workspace sizes, shape and type checks of the wrappers."""
import pytest
import torch

import w4_gemm_amd as W
from w4_gemm_amd import _lib
from w4_gemm_amd import shapes as S


def _payload(n=200, k=300, codes=0x1000, exps=0x2000):
    return _lib.SqF8(n, k, codes, exps)


# no call has a workspace: what is not refused for another reason is refused for that one
def _calls(p, up=None, m=4, a=0x8000, out=0x9000, dt=0, act=0, ws=0xA000, nb=0, offsets=0xB000, groups=2,
           g=0xC000, u=0xD000, dg=0xE000, du=0xF000):
    up = p if up is None else up
    return [_lib.sq_linear_fwd_f8(a, m, p, out, dt, ws, nb, None),
            _lib.sq_linear_dgrad_f8(a, m, p, out, dt, ws, nb, None),
            _lib.sq_grouped_fwd_f8(a, m, offsets, groups, p, out, dt, ws, nb, None),
            _lib.sq_grouped_dgrad_f8(a, m, offsets, groups, p, out, dt, ws, nb, None),
            _lib.sq_gated_fwd_f8(a, m, p, up, act, out, dt, g, u, ws, nb, None),
            _lib.sq_gated_bwd_f8(a, g, u, m, p, up, act, out, dt, dg, du, ws, nb, None),
            _lib.sq_grouped_gated_fwd_f8(a, m, offsets, groups, p, up, act, out, dt, g, u, ws, nb, None),
            _lib.sq_grouped_gated_bwd_f8(a, g, u, m, offsets, groups, p, up, act, out, dt, dg, du, ws, nb, None)]


ALL, GATED = 8, 4


@pytest.mark.parametrize("kw,status", [
    (dict(n=0), 2), (dict(k=0), 2), (dict(n=-1), 2), (dict(n=(1 << 20) + 1), 2), (dict(k=(1 << 20) + 1), 2),
    (dict(codes=None), 1), (dict(exps=None), 1), (dict(codes=0x1008), 5), (dict(exps=0x2004), 5),
], ids=str)
def test_payload_is_refused(kw, status):
    assert _calls(_payload(**kw)) == [status] * ALL
    assert _calls(_payload(), up=_payload(**kw))[GATED:] == [status] * GATED
    assert _lib.sq_quantize_weight_f8(0x6000, 0, _payload(**kw), 0x7000, None) == status


def test_arguments_are_refused():
    p = _payload()
    assert _calls(p, m=-1) == [2] * ALL
    assert _calls(p, m=1 << 31) == [2] * ALL
    assert _calls(p, dt=2) == [7] * ALL
    assert _calls(p, dt=-1) == [7] * ALL
    assert _calls(p, a=None) == [1] * ALL
    assert _calls(p, out=None) == [1] * ALL
    assert _calls(p, ws=None) == [1] * ALL
    assert _calls(p, a=0x8004) == [5] * ALL
    assert _calls(p, out=0x9008) == [5] * ALL
    assert _calls(p, ws=0xA001) == [5] * ALL
    assert _calls(p, nb=0) == [6] * ALL
    assert _calls(p, m=0, a=None, out=None, ws=None, nb=0, offsets=None, g=None, u=None) == [0] * ALL
    grouped = [False, False, True, True, False, False, True, True]
    for kw, status in ((dict(offsets=None), 1), (dict(offsets=0xB004), 5), (dict(groups=0), 2), (dict(groups=-3), 2)):
        got = _calls(p, nb=0, **kw)
        assert got == [status if is_grouped else 6 for is_grouped in grouped]
    assert [s for s, is_grouped in zip(_calls(p, m=1 << 30, groups=1 << 20), grouped) if is_grouped] == [2] * 4


def test_gated_arguments_are_refused():
    p = _payload()
    for act in (-1, 3):
        assert _calls(p, nb=0, act=act) == [6] * GATED + [10] * GATED
    for up in (_payload(n=201), _payload(k=301)):
        assert _calls(p, nb=0, up=up) == [6] * GATED + [2] * GATED
    assert _lib.sq_gated_fwd_f8(0x8000, 4, p, None, 0, 0x9000, 0, None, None, 0xA000, 0, None) == 1
    # the forward saves both or neither; the backward needs both and writes either
    fwd = [4, 6]
    for kw in (dict(g=None), dict(u=None)):
        assert [_calls(p, nb=0, **kw)[i] for i in range(GATED, ALL)] == [1] * GATED
    got = _calls(p, nb=0, g=None, u=None)
    assert [got[i] for i in fwd] == [6, 6] and [got[i] for i in (5, 7)] == [1, 1]
    for kw in (dict(g=0xC002), dict(u=0xD008)):
        assert _calls(p, nb=0, **kw)[GATED:] == [5] * GATED
    for kw in (dict(dg=0xE004), dict(du=0xF004)):
        assert _calls(p, nb=0, **kw)[GATED:] == [6, 5, 6, 5]
    for kw in (dict(dg=None), dict(du=None), dict(dg=None, du=None)):
        assert _calls(p, nb=0, **kw)[GATED:] == [6] * GATED


def test_quantizer_arguments():
    p = _payload()
    q = _lib.sq_quantize_weight_f8
    assert q(0x6000, 2, p, 0x7000, None) == 7
    assert q(None, 0, p, 0x7000, None) == 1
    assert q(0x6000, 0, p, None, None) == 1
    assert q(0x6004, 0, p, 0x7000, None) == 5
    assert q(0x6000, 1, p, 0x7004, None) == 5
    assert q(0x6000, 0, _payload(n=1 << 20, k=1 << 20), 0x7000, None) == 2      # 2^26 blocks


def _sizes(m, p, groups=None):
    if groups is None:
        return [_lib.sq_linear_fwd_f8_workspace_bytes(m, p), _lib.sq_linear_dgrad_f8_workspace_bytes(m, p),
                _lib.sq_gated_fwd_f8_workspace_bytes(m, p), _lib.sq_gated_bwd_f8_workspace_bytes(m, p)]
    return [_lib.sq_grouped_fwd_f8_workspace_bytes(m, groups, p), _lib.sq_grouped_dgrad_f8_workspace_bytes(m, groups, p),
            _lib.sq_grouped_gated_fwd_f8_workspace_bytes(m, groups, p),
            _lib.sq_grouped_gated_bwd_f8_workspace_bytes(m, groups, p)]


def test_workspace_bytes():
    p = _payload(n=200, k=500)
    for m in (1, 16, 17, 300, 5000):
        one = _sizes(m, p)
        assert _sizes(m, p, 1) == one
        order = [0, 1, 0, 1, 2, 3, 2, 3]       # size of each call of _calls
        for i, nb in enumerate(one):
            assert nb > 0
            for dt in (0, 1):
                got = _calls(p, m=m, dt=dt, nb=0, groups=1)
                assert [got[c] for c in range(ALL) if order[c] == i] == [6, 6]
    for m, groups in ((0, 1), (-1, 1), (4, 0), (1 << 31, 1), (1 << 30, 1 << 20)):
        assert _sizes(m, p, groups) == [0] * 4
    assert _sizes(4, _payload(n=0)) == [0] * 4 and _sizes(4, _payload(k=(1 << 20) + 1)) == [0] * 4


def test_launches_past_two_to_the_32_threads_are_refused():
    p = _payload(n=1 << 20, k=128)
    m = 1 << 22
    sizes = _sizes(m, p)
    assert sizes[0] == 0 and sizes[2] == 0           # 2^22 x 2^20 results
    assert _calls(p, m=m)[0] == 2 and _calls(p, m=m)[4] == 2
    assert all(_sizes(1 << 20, _payload(n=256, k=256)))


def test_status_text():
    assert "activation" in _lib.status_str(10)
    assert "2^20" in _lib.status_str(2)


# ------------------------------------------------------------------ wrappers
def _tensors(n=8, k=200, e=None):
    lead = () if e is None else (e,)
    codes = torch.zeros((*lead, n, 256), dtype=torch.uint8).view(torch.float8_e4m3fn)
    exps = torch.zeros((*lead, -(-n // 128), 2), dtype=torch.uint8)
    return W.F8Payload(codes, exps, k) if e is None else W.GroupedF8Payload(codes, exps, k)


def test_payload_shapes():
    assert S.check_f8_payload((8, 256), (1, 2), 200) == (8, 200)
    assert S.check_f8_payload((129, 128), (2, 1), 1) == (129, 1)
    assert S.check_grouped_f8_payload((3, 8, 256), (3, 1, 2), 129) == (3, 8, 129)
    for codes, exps, k in (((8, 200), (1, 2), 200), ((8, 256), (1, 1), 200), ((8, 256), (2, 2), 200),
                           ((8, 256), (1, 2), 128), ((8, 256), (1, 2), 257), ((8, 256), (1, 2), 0),
                           ((0, 256), (0, 2), 200), ((8,), (1, 2), 200), ((3, 8, 256), (1, 2), 200),
                           ((1, 1 << 21), (1, 1 << 14), 1 << 21)):
        with pytest.raises(ValueError):
            S.check_f8_payload(codes, exps, k)
    for codes, exps in (((8, 256), (1, 2)), ((0, 8, 256), (0, 1, 2)), ((3, 8, 256), (2, 1, 2)), ((3, 8, 256), (3, 2))):
        with pytest.raises(ValueError):
            S.check_grouped_f8_payload(codes, exps, 200)


def test_payload_accessors_and_stack():
    one = _tensors()
    many = W.stack_payloads_f8([one, one, one])
    assert (one.n, one.k, many.groups, many.n, many.k) == (8, 200, 3, 8, 200)
    assert W.empty_payload_f8(130, 129, device="cpu").codes.shape == (130, 256)
    with pytest.raises(ValueError):
        W.stack_payloads_f8([])
    with pytest.raises(ValueError):
        W.stack_payloads_f8([one, _tensors(n=9)])
    with pytest.raises(TypeError):
        W.stack_payloads_f8([many])


X, DY = torch.zeros((4, 200), dtype=torch.bfloat16), torch.zeros((4, 8), dtype=torch.bfloat16)
OFF = torch.tensor([0, 1, 2, 4], dtype=torch.int32)


@pytest.mark.parametrize("call", [
    lambda p: W.linear_fwd_f8(X, p), lambda p: W.linear_dgrad_f8(DY, p), lambda p: W.gated_fwd_f8(X, p, p),
    lambda p: W.gated_bwd_f8(DY, DY, DY, p, p), lambda p: W.fwd_f8_workspace_bytes(4, p),
    lambda p: W.dgrad_f8_workspace_bytes(4, p), lambda p: W.gated_fwd_f8_workspace_bytes(4, p),
    lambda p: W.gated_bwd_f8_workspace_bytes(4, p), lambda p: W.gated_fwd_f8(X, _tensors(), p),
])
def test_calls_for_one_layer_refuse_a_stack(call):
    for p in (_tensors(e=3), W.W8Payload(None, None, None, None)):
        with pytest.raises(TypeError, match="F8Payload"):
            call(p)


@pytest.mark.parametrize("call", [
    lambda p: W.grouped_fwd_f8(X, OFF, p), lambda p: W.grouped_dgrad_f8(DY, OFF, p),
    lambda p: W.grouped_gated_fwd_f8(X, OFF, p, p), lambda p: W.grouped_gated_bwd_f8(DY, DY, DY, OFF, p, p),
    lambda p: W.grouped_fwd_f8_workspace_bytes(4, p), lambda p: W.grouped_dgrad_f8_workspace_bytes(4, p),
    lambda p: W.grouped_gated_fwd_f8_workspace_bytes(4, p), lambda p: W.grouped_gated_bwd_f8_workspace_bytes(4, p),
])
def test_grouped_calls_refuse_one_layer(call):
    with pytest.raises(TypeError, match="GroupedF8Payload"):
        call(_tensors())


def test_pairs_and_activations_are_checked():
    p = _tensors()
    with pytest.raises(ValueError, match="same shape"):
        W.gated_fwd_f8(X, p, _tensors(n=9))
    with pytest.raises(ValueError, match="same shape"):
        W.gated_bwd_f8(DY, DY, DY, p, _tensors(k=201))
    for act in ("relu", None, 0):
        with pytest.raises(ValueError, match="act"):
            W.gated_fwd_f8(X, p, p, act)
