"""What the norms' calls refuse, before anything is launched: no GPU is needed."""
import ctypes

import pytest
import torch

P = [0x100000 + 0x100000 * i for i in range(16)]


@pytest.fixture(scope="module")
def lib():
    from exact_attention_67_gb300 import build as b
    b.build()
    from exact_attention_67_gb300 import _lib
    return _lib.load()


def S(B=1, H=2, N=16, d=64):
    from exact_attention_67_gb300 import Strides
    return Strides(H * N * d, N * d, d)


def norm(lib, dtype=0, q=P[0], qo=P[1], Hq=2, k=P[2], ko=P[3], Hk=2, pos=P[4], ps=0, freq=P[5], rot=64, factor=1.0, qg=P[6], kg=P[7],
         gtype=2, eps=1e-6, B=1, N=16, d=64, sq=None):
    s = S()
    return lib.attn_norm_rotary(dtype, q, sq or s, qo, s, Hq, k, s, ko, s, Hk, pos, ps, freq, rot, 0, factor, qg, kg, gtype, eps, B, N, d,
                                None)


def grad(lib, dq=P[8], dk=P[9], ws=P[10], ws_bytes=1 << 20, dqg=P[11], dkg=P[12], gtype=2, eps=1e-6, sdq=None, N=16, Hk=2, d=64):
    s = S()
    return lib.attn_norm_rotary_backward(0, dq, sdq or s, P[0], s, P[1], s, 2, dk, s, P[2], s, P[3], s, Hk, P[4], 0, P[5], 64, 0, 1.0, P[6],
                                         P[7], gtype, eps, dqg, dkg, 1, N, d, ws, ws_bytes, None)


NULL, SHAPE, ALIGN, UNSUPPORTED, WORKSPACE, VALUE = 1, 2, 3, 4, 6, 9


@pytest.mark.parametrize("how,status", [
    (dict(q=None), NULL), (dict(qo=None), NULL), (dict(ko=None), NULL), (dict(pos=None), NULL), (dict(freq=None), NULL),
    (dict(dtype=2), UNSUPPORTED), (dict(d=96), UNSUPPORTED), (dict(rot=3), UNSUPPORTED), (dict(rot=66), UNSUPPORTED),
    (dict(gtype=3), UNSUPPORTED), (dict(gtype=-1), UNSUPPORTED), (dict(Hq=0), SHAPE), (dict(N=0), SHAPE), (dict(ps=-1), SHAPE),
    (dict(q=P[0] + 8), ALIGN), (dict(qg=P[6] + 2), ALIGN), (dict(qg=P[6] + 1, gtype=0), ALIGN), (dict(kg=P[7] + 2), ALIGN),
    (dict(eps=-1e-6), VALUE), (dict(eps=float("nan")), VALUE), (dict(eps=float("inf")), VALUE), (dict(factor=0.0), VALUE)])
def test_refusals(lib, how, status):
    assert norm(lib, **how) == status


@pytest.mark.parametrize("how,status", [
    (dict(dq=None), NULL), (dict(dk=None), NULL), (dict(ws=None), WORKSPACE), (dict(ws_bytes=16 * 2 * 64 * 4 - 1), WORKSPACE),
    (dict(ws=P[10] + 8), ALIGN), (dict(dq=P[8] + 8), ALIGN), (dict(dqg=P[11] + 2), ALIGN), (dict(gtype=7), UNSUPPORTED),
    (dict(eps=-1.0), VALUE), (dict(N=0), SHAPE), (dict(d=32), UNSUPPORTED)])
def test_gradient_refusals(lib, how, status):
    assert grad(lib, **how) == status


def test_gradient_strides(lib):
    from exact_attention_67_gb300 import Strides
    assert grad(lib, sdq=Strides(2048, 1024, 63)) == ALIGN
    assert grad(lib, sdq=Strides(2048, 1024, 0)) == SHAPE


def test_workspace_size(lib):
    size = lib.attn_norm_rotary_backward_workspace_size
    size.restype = ctypes.c_size_t
    assert size(1, 1, 64) == 2 * 64 * 4 and size(2, 8, 128) == 16 * 2 * 128 * 4
    assert size(8, 1 << 20, 128) == size(1, 1 << 20, 128) < 1 << 20  # a bounded number of blocks
    assert size(0, 8, 64) == size(1, 0, 64) == size(1, 8, 96) == size(1 << 16, 1 << 16, 64) == 0


def append(lib, **how):
    a = dict(q=P[0], qo=P[1], Hq=2, freq=P[5], rot=64, qg=P[6], kg=P[7], gtype=0, eps=1e-6)
    a.update(how)
    s = S()
    return lib.attn_cache_append_norm(0, a["q"], s, a["qo"], s, a["Hq"], P[2], s, P[3], s, P[8], s, P[9], s, 2, 4, 16, P[10], 4, 4, P[11],
                                      None, 1, 16, 64, a["freq"], a["rot"], 0, 1.0, a["qg"], a["kg"], a["gtype"], a["eps"], None)


@pytest.mark.parametrize("how,status", [
    (dict(qo=None), NULL), (dict(gtype=5), UNSUPPORTED), (dict(kg=P[7] + 1), ALIGN), (dict(eps=-1.0), VALUE), (dict(rot=5), UNSUPPORTED),
    (dict(q=P[0] + 2), ALIGN)])
def test_append_refusals(lib, how, status):
    assert append(lib, **how) == status


def test_python_refusals():
    import exact_attention_67_gb300 as ex
    from exact_attention_67_gb300 import build
    build.build()
    q, g = torch.zeros(1, 2, 4, 64, dtype=torch.bfloat16), torch.ones(64)
    pos, freq = torch.arange(4, dtype=torch.int32), ex.rotary_frequencies(64, device="cpu")[0]
    with pytest.raises(ValueError, match="CUDA"):
        ex.norm_rotary(q, q, g, g, pos, freq)
    with pytest.raises(ValueError, match="CUDA"):
        ex.norm_rotary_backward(q, q, q, q, g, g, pos, freq)
    with pytest.raises(TypeError):
        ex.norm_rotary(q.float(), None, g, None, pos, freq)
    with pytest.raises((TypeError, ValueError)):
        ex.norm_rotary_backward(None, None, q, None, g, None, pos, freq)
    with pytest.raises(ValueError, match="current stream"):
        ex.norm_rotary(q.requires_grad_(), q, g, g, pos, freq, stream=0)
