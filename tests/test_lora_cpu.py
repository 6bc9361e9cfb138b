"""The adapter calls refuse what they cannot do, before anything is launched:
the C ABI's checks (no pointer below is followed) and the binding's."""
import ctypes

import pytest
import torch

from lm_head_fp32_b200 import decode, lmhead, loss

P = ctypes.c_void_p
A = P(0x10000)
INVALID, MISALIGNED, UNSUPPORTED = (lmhead.LMH_ERR_INVALID_ARG, lmhead.LMH_ERR_MISALIGNED,
                                    lmhead.LMH_ERR_UNSUPPORTED)
DIMS = dict(M=16, K=64, V=64, R=16, N=4)
GEMM = ["X", "W", "A", "B", "scale", "adapter", "t", "out"]
GRAD = ["dl", "X", "u", "g", "adapter", "dA", "dB"]


def gemm(fn, **kw):
    a = dict({k: A for k in GEMM}, dtype=lmhead.F32, ws=A, nbytes=1 << 40, **DIMS)
    a.update(kw)
    return getattr(lmhead.lib(), fn)(*a.values(), None, None)


def grad(**kw):
    a = dict({k: A for k in GRAD}, ws=A, nbytes=1 << 40, **DIMS)
    a.update(kw)
    return lmhead.lib().lmhead_bwd_lora(*a.values(), None, None)


BAD_DIMS = [dict(M=0), dict(K=0), dict(V=0), dict(R=0), dict(N=0), dict(R=264), dict(N=65536),
            dict(M=65535 * 64 + 1), dict(M=1 << 20, N=1 << 15), dict(V=1 << 31), dict(nbytes=1000)]


@pytest.mark.parametrize("fn", ["lmhead_fwd_lora", "lmhead_bwd_dx_lora"])
def test_gemm_calls(fn):
    for kw in BAD_DIMS + [{k: None} for k in GEMM + ["ws"]]:
        assert gemm(fn, **kw) == INVALID, kw
    assert gemm(fn, dtype=lmhead.F16) == UNSUPPORTED
    for kw in [dict(K=60), dict(R=12), dict(ws=P(0x10010))] + \
            [{k: P(0x10008)} for k in ("X", "W", "A", "B")] + \
            [{k: P(0x10002)} for k in ("scale", "adapter", "t", "out")]:
        assert gemm(fn, **kw) == MISALIGNED, kw
    if fn == "lmhead_bwd_dx_lora":
        assert gemm(fn, V=100) == MISALIGNED
        assert gemm(fn, out=P(0x10008)) == MISALIGNED


def test_grad_call():
    for kw in BAD_DIMS + [{k: None} for k in GRAD + ["ws"]]:
        assert grad(**kw) == INVALID, kw
    for kw in [dict(K=60), dict(V=100), dict(R=12), dict(ws=P(0x10010))] + \
            [{k: P(0x10008)} for k in ("dl", "X", "dA", "dB")] + \
            [{k: P(0x10002)} for k in ("u", "g", "adapter")]:
        assert grad(**kw) == MISALIGNED, kw


def test_workspace_bytes():
    f = lmhead.lmhead_lora_workspace_bytes
    assert f(0, 64, 64, 16, 1) == f(1, 64, 64, 0, 1) == f(1, 64, 64, 264, 1) == f(1, 64, 64, 8, 0) == -1
    assert f(65535 * 64 + 1, 64, 64, 16, 1) == -1
    # room for the split u of every token tile, and for the gradient call's parts
    for M in (1, 17, 300, 4096):
        assert f(M, 4096, 32768, 16, 8) >= M * 128 and f(M, 64, 64, 16, 8) >= 2 * M * 3 * 16 * 2


def _args(M=4, K=16, V=24, R=8, N=2):
    b = torch.bfloat16
    return [torch.zeros(M, K, dtype=b), torch.zeros(V, K, dtype=b), torch.zeros(N, R, K, dtype=b),
            torch.zeros(N, V, R, dtype=b), torch.ones(N), torch.zeros(M, dtype=torch.int32),
            torch.zeros(M, R), torch.zeros(M, V), torch.zeros(1 << 16, dtype=torch.uint8)]


def test_binding_refuses():
    with pytest.raises(ValueError, match="CUDA"):
        lmhead.lmhead_fwd_lora(*_args())
    for i, bad in ((0, torch.zeros(4, 16)), (1, torch.zeros(24, 8, dtype=torch.bfloat16)),
                   (2, torch.zeros(2, 16, 8, dtype=torch.bfloat16).transpose(1, 2)),
                   (3, torch.zeros(2, 8, 24, dtype=torch.bfloat16)), (4, torch.ones(3)),
                   (5, torch.zeros(4, dtype=torch.int64)), (5, torch.zeros(5, dtype=torch.int32)),
                   (6, torch.zeros(4, 16)), (7, torch.zeros(4, 24).half())):
        a = _args()
        a[i] = bad
        with pytest.raises((ValueError, TypeError)):
            lmhead.lmhead_fwd_lora(*a)
    X, W, A_, B, s, ids = _args()[:6]
    t = torch.zeros(4, dtype=torch.int64)
    with pytest.raises(ValueError, match="CUDA"):
        loss.lm_head_lora_cross_entropy(X, W, A_, B, s, ids, t)


def test_decoder_refuses():
    W = torch.zeros(24, 16, dtype=torch.bfloat16)
    A_, B, s = _args()[2:5]
    with pytest.raises(ValueError, match="together"):
        decode.BeamDecoder(W, 2, 2, A=A_, B=B)
    with pytest.raises(ValueError, match="out of range"):
        decode.BeamDecoder(W, 2, 65)
    with pytest.raises(ValueError, match="out of range"):
        decode.BeamDecoder(W, 2, 2, A=torch.zeros(2, 300, 16), B=B, scale=s)
    d = decode.BeamDecoder(W, 2, 2, eos=3, A=A_, B=B, scale=s)
    assert d.scores.tolist() == [[0.0, float("-inf")]] * 2
    with pytest.raises(ValueError, match="adapter ids"):
        d.step(torch.zeros(4, 16, dtype=torch.bfloat16))
