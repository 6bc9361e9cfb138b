"""beam_select and beam_reorder refuse what they cannot do, before anything is
launched: the C ABI's checks (no pointer below is followed) and the binding's."""
import ctypes

import pytest
import torch

from lm_head_fp32_b200 import lmhead

P = ctypes.c_void_p
A = P(0x10000)
ODD = P(0x10002)
INVALID, MISALIGNED, UNSUPPORTED = (lmhead.LMH_ERR_INVALID_ARG, lmhead.LMH_ERR_MISALIGNED,
                                    lmhead.LMH_ERR_UNSUPPORTED)


def select(**kw):
    a = dict(logits=A, dtype=lmhead.F32, scores=A, done=None, cs=A, cb=A, ct=A, ns=A, nb=A, nt=A,
             ws=A, nbytes=1 << 40, N=2, W=4, V=1000, C=8, eos=2)
    a.update(kw)
    return lmhead.lib().beam_select(*a.values(), None, None)


@pytest.mark.parametrize("kw", [
    dict(logits=None), dict(scores=None), dict(cs=None), dict(cb=None), dict(ct=None), dict(ws=None),
    dict(ns=None), dict(nt=None),                  # next_*: all three or none
    dict(N=0), dict(W=0), dict(V=0), dict(C=0), dict(W=65, C=128), dict(C=129), dict(V=1 << 31),
    dict(N=1 << 30), dict(eos=-2), dict(eos=1000),
    dict(C=7), dict(C=3, eos=-1),                  # too few candidates for W that go on
    dict(nbytes=100),
])
def test_select_invalid(kw):
    assert select(**kw) == INVALID


def test_select_unsupported_and_misaligned():
    assert select(dtype=lmhead.F16) == UNSUPPORTED
    assert select(logits=ODD) == MISALIGNED
    for k in ("scores", "done", "cs", "cb", "ns", "nb"):
        assert select(**{k: ODD}) == MISALIGNED, k
    assert select(ct=P(0x10004)) == MISALIGNED
    assert select(nt=P(0x10004)) == MISALIGNED
    assert select(ws=P(0x10008)) == MISALIGNED


def test_select_workspace_bytes():
    f = lmhead.beam_select_workspace_bytes
    assert f(1, 1, 1, 1) == 16 + 8
    assert f(3, 2, 4097, 4) == 3 * 2 * 2 * (16 + 8 * 4)
    assert f(0, 1, 1, 1) == f(1, 65, 1, 1) == f(1, 1, 1, 129) == f(1, 1, 1 << 31, 1) == -1
    # the scan's CTAs, at least one per row and 65536 logits, are counted in 32 bits
    assert f(1 << 20, 64, (1 << 31) - 1, 128) == -1 < f(1, 64, (1 << 31) - 1, 128)


def reorder(states=(0x10000,), parents=A, N=2, W=4, es=4096, bs=1024, run=64, outer=(16,), os=(64,)):
    ptrs = (P * len(states))(*states) if states else None
    k = len(outer)
    I = ctypes.c_int64
    return lmhead.lib().beam_reorder(ptrs, len(states), parents, N, W, es, bs, run, (I * k)(*outer),
                                     (I * k)(*os), k, None, None)


@pytest.mark.parametrize("kw", [
    dict(states=()), dict(states=(None,)), dict(states=tuple(0x10000 + 16 * i for i in range(129))),
    dict(states=(0x10000, 0x20000, 0x10000)),       # a state given twice
    dict(parents=None), dict(N=0), dict(W=0), dict(W=65), dict(N=65536), dict(run=0),
    dict(outer=(1, 1, 1, 1), os=(0, 0, 0, 0)), dict(outer=(0,)), dict(outer=(1 << 31,)),
    dict(bs=0), dict(bs=-1024), dict(es=0), dict(os=(0,)), dict(os=(-64,)),
    dict(os=(32,)),                                  # steps by less than the run
    dict(bs=512), dict(es=2048),                     # beams and entries overlap
    dict(outer=(16, 3), os=(64, 2048)),
    dict(es=1 << 60), dict(run=1 << 50, es=1 << 54, bs=1 << 52, outer=()),
    dict(run=1 << 40, bs=1 << 41, es=1 << 43, outer=()),   # more columns than 32 bits
])
def test_reorder_invalid(kw):
    if kw.get("outer") == ():
        kw["os"] = ()
    assert reorder(**kw) == INVALID


def test_reorder_parents_alignment():
    assert reorder(parents=ODD) == MISALIGNED


def _args(N=2, W=3, V=50, C=6):
    f = torch.float32
    return [torch.zeros(N, W, V), torch.zeros(N, W), torch.zeros(N, C),
            torch.zeros(N, C, dtype=torch.int32), torch.zeros(N, C, dtype=torch.int64),
            torch.zeros(N, W, dtype=f), torch.zeros(N, W, dtype=torch.int32),
            torch.zeros(N, W, dtype=torch.int64), torch.zeros(4096, dtype=torch.uint8)]


def test_binding_select_refuses():
    with pytest.raises(ValueError, match="CUDA"):      # no CPU path
        lmhead.beam_select(*_args())
    for i, bad in ((1, torch.zeros(3, 2)), (3, torch.zeros(2, 6, dtype=torch.int64)),
                   (4, torch.zeros(2, 6, dtype=torch.int32)), (0, torch.zeros(2, 3, 50).half()),
                   (0, torch.zeros(6, 50)), (0, torch.zeros(2, 50, 3).transpose(1, 2)),
                   (7, torch.zeros(2, 2, dtype=torch.int64))):
        a = _args()
        a[i] = bad
        with pytest.raises((ValueError, TypeError)):
            lmhead.beam_select(*a)
    with pytest.raises(ValueError):
        lmhead.beam_select(*_args(), done=torch.zeros(3, dtype=torch.int32))


def test_binding_reorder_refuses():
    par = torch.zeros(2, 3, dtype=torch.int32)
    for states, kw in (([], {}), ([torch.zeros(2, 4, 5)], {}), ([torch.zeros(2, 3)], dict(entry_dim=1)),
                       ([torch.zeros(2, 3, 5), torch.zeros(2, 3, 6)], {}),
                       ([torch.zeros(2, 3, 5), torch.zeros(2, 3, 5).double()], {}),
                       # five strided dimensions beside the beams
                       ([torch.zeros(2, 3, 3, 3, 3, 3, 3)[:, :, :2, :2, :2, :2, :2]], {})):
        with pytest.raises(ValueError):
            lmhead.beam_reorder(states, par, **kw)
    with pytest.raises(ValueError, match="CUDA"):
        lmhead.beam_reorder(torch.zeros(2, 3, 5), par)
    with pytest.raises(TypeError):
        lmhead.beam_reorder(torch.zeros(2, 3, 5), par.long())


def test_state_geometry():
    def g(t, entry_dim):
        run, outer, strides = lmhead._state_geometry(tuple(t.shape), t.stride(), t.element_size(), entry_dim)
        return run, list(outer), list(strides)
    t = torch.zeros(2, 4, 3, 8, 16, 6)                          # [outer, N, W, heads, room, width]
    assert g(t[:, :, :, :, :10], 1) == (10 * 6 * 4, [8, 2], [16 * 6 * 4, 4 * 3 * 8 * 16 * 6 * 4])
    assert g(t, 1) == (8 * 16 * 6 * 4, [2], [4 * 3 * 8 * 16 * 6 * 4])
    assert g(torch.zeros(4, 3), 0) == (4, [], [])
    assert g(torch.zeros(7, 4, 3, dtype=torch.int64).permute(1, 2, 0), 0) == (8, [7], [96])
