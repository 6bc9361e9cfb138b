"""beam_reorder refuses states that share memory, and takes those that only lie between each
other's rows; a decoder over a vocabulary of one token; entries that are done."""
import ctypes
import itertools
import random

import pytest
import torch

from lm_head_fp32_b200 import decode, lmhead

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


def decoder(V, eos, device, E=2, beams=2, K=16):
    W = torch.ones((V, K), dtype=torch.bfloat16, device=device)
    return decode.BeamDecoder(W, E, beams, eos=eos)


def test_decoder_buffers_of_a_vocabulary_of_one_token():
    for eos in (-1, 0):
        d = decoder(1, eos, "cpu")
        assert d.cand_score.shape == d.cand_beam.shape == d.cand_token.shape == (2, 4)


@pytest.mark.gpu
def test_decoder_over_a_vocabulary_of_one_token():
    inf = float("inf")
    X = torch.ones((4, 16), dtype=torch.bfloat16, device="cuda")
    d = decoder(1, 0, "cuda")
    tokens, parents, scores = d.step(X)
    # its one token ends every sequence
    assert d.cand_score.tolist() == [[0.0, -inf, -inf, -inf]] * 2
    assert d.cand_token.tolist() == [[0, -1, -1, -1]] * 2 and scores.tolist() == [[-inf, -inf]] * 2
    d = decoder(1, -1, "cuda")
    for _ in range(3):
        tokens, parents, scores = d.step(X)
        assert scores.tolist() == [[0.0, -inf]] * 2 and parents.tolist() == [[0, 1]] * 2
    assert int(d.status.item()) == 0


@pytest.mark.gpu
def test_decoder_leaves_entries_that_are_done():
    E, beams, K, V = 3, 4, 64, 500
    gen = torch.Generator().manual_seed(2)
    W = torch.randn((V, K), generator=gen).to(torch.bfloat16).cuda()
    a, b = (decode.BeamDecoder(W, E, beams, eos=7) for _ in range(2))
    hist = [torch.arange(E * beams * 5, device="cuda").view(E, beams, 5).clone() for _ in range(2)]
    done = torch.tensor([0, 1, 0], dtype=torch.int32, device="cuda")
    for step in range(3):
        X = torch.randn((E * beams, K), generator=gen).to(torch.bfloat16).cuda()
        before, kept = b.scores.clone(), hist[1][1].clone()
        a.step(X, hist[0])
        b.step(X, hist[1], done=done if step else None)
        for e in (0, 2):
            for f in ("tokens", "parents", "scores", "cand_score", "cand_beam", "cand_token"):
                assert torch.equal(getattr(a, f)[e], getattr(b, f)[e])
            assert torch.equal(hist[0][e], hist[1][e])
        if step:
            assert torch.equal(b.scores[1], before[1]) and torch.equal(hist[1][1], kept)
            assert b.parents[1].tolist() == [0, 1, 2, 3] and b.cand_beam[1].tolist() == [-1] * 8
            assert b.tokens[1].tolist() == [7] * 4
    assert int(b.status.item()) == 0
