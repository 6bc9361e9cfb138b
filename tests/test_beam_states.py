"""beam_reorder refuses states that share memory, and takes those that only lie between each
other's rows; a decoder over a vocabulary of one token; entries that are done."""
import ctypes
import itertools
import random

import pytest
import torch

from lm_head_fp32_b200 import lmhead

P = ctypes.c_void_p
BASE = 0x10000000


def call(states, N, W, es, bs, run, outer, strides):
    """The C call; refused calls launch nothing (no pointer is followed)."""
    I, k = ctypes.c_int64, len(outer)
    return lmhead.lib().beam_reorder((P * len(states))(*states), len(states), P(0x10000), N, W, es, bs, run,
                                     (I * k)(*outer), (I * k)(*strides), k, None, None)


def covered(N, W, es, bs, run, outer, strides):
    """Every byte of a state, as offsets."""
    dims = [(N, es), (W, bs)] + list(zip(outer, strides))
    return {sum(i * s for i, (_, s) in zip(at, dims)) + b
            for at in itertools.product(*(range(n) for n, _ in dims)) for b in range(run)}


def geometry(rng):
    """A random state: dimensions in a random order, each over all below it with some room."""
    run = rng.choice([1, 2, 4, 6, 16])
    names = ["N", "W"] + list(range(rng.randint(0, 3)))
    rng.shuffle(names)
    ext, stride, span = {}, {}, run
    for k in names:
        ext[k] = rng.randint(1, 3)
        stride[k] = span + rng.choice([0, 0, 1, 3, run, 2 * run, span])
        span += (ext[k] - 1) * stride[k]
    outer = [k for k in names if k not in ("N", "W")]
    return ext["N"], ext["W"], stride["N"], stride["W"], run, [ext[k] for k in outer], [stride[k] for k in outer]


def pairs(seed, n):
    """Random geometries with a distance of two states: (geometry, distance, whether they share)."""
    rng = random.Random(seed)
    for _ in range(n):
        geo = geometry(rng)
        own = covered(*geo)
        d = rng.randint(1, max(own) + 2)
        yield geo, d, bool(own & {o + d for o in own})


def test_states_that_share_memory_are_refused():
    sharing = [(geo, d) for geo, d, share in pairs(1, 3000) if share]
    assert len(sharing) > 500
    for geo, d in sharing:
        for two in ((BASE, BASE + d), (BASE + d, BASE)):
            assert call(two, *geo) == lmhead.LMH_ERR_INVALID_ARG, (geo, d)
        assert call((BASE, 2 * BASE, BASE + d), *geo) == lmhead.LMH_ERR_INVALID_ARG


@pytest.mark.gpu
def test_states_between_each_others_rows_are_taken():
    between = [(geo, d) for geo, d, share in pairs(2, 1500) if not share and d <= max(covered(*geo))]
    assert len(between) > 60
    gen = torch.Generator().manual_seed(1)
    for (N, W, es, bs, run, outer, strides), d in between[:120]:
        size = (N, W, *outer, run)
        step = (es, bs, *strides, 1)
        end = sum((n - 1) * s for n, s in zip(size, step)) + 1 + d
        host = torch.randint(0, 256, (end,), generator=gen, dtype=torch.int64).to(torch.uint8)
        dev = host.cuda()
        par = torch.randint(0, W, (N, W), generator=gen, dtype=torch.int32)
        views = [dev.as_strided(size, step, o) for o in (0, d)]
        ptrs = tuple(v.data_ptr() for v in views)
        gpu_par = par.cuda()
        I, k = ctypes.c_int64, len(outer)
        code = lmhead.lib().beam_reorder((P * 2)(*ptrs), 2, P(gpu_par.data_ptr()), N, W, es, bs, run,
                                         (I * k)(*outer), (I * k)(*strides), k, None,
                                         torch.cuda.current_stream().cuda_stream)
        assert code == lmhead.LMH_OK
        want = host.clone()
        for o in (0, d):
            old, new = host.as_strided(size, step, o), want.as_strided(size, step, o)
            for n in range(N):
                for w in range(W):
                    new[n, w] = old[n, int(par[n, w])]
        assert torch.equal(dev.cpu(), want)


@pytest.mark.gpu
def test_views_that_share_rows_are_refused():
    cache = torch.zeros((2, 3, 40, 8), device="cuda")
    par = torch.zeros((2, 3), dtype=torch.int32, device="cuda")
    with pytest.raises(lmhead.LmhError):
        lmhead.beam_reorder([cache[:, :, :30], cache[:, :, 10:]], par)
    lmhead.beam_reorder([cache[:, :, :20], cache[:, :, 20:]], par)
