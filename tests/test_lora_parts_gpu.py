"""The adapters' factor u (g) keeps FP32's bits in the second product, whatever the type of
the output: exact cases, where a factor held in 16 bits, a lost or a misplaced part shows.

Every u is a whole number of 22 bits times a power of two, made of three BF16 features; B has
one value per row.  So each logit's adapter term is one product with a power of two, and
where W takes away the two upper features' share, the logit is the third feature's alone, of 6
bits.  All sums are whole numbers below 2^24 times one power of two: exact in FP32 in any
order, and every result below is compared for equality.
"""
import pytest
import torch

from lm_head_fp32_b200 import lmhead
from helpers import guarded_empty

pytestmark = pytest.mark.gpu
DEV = "cuda"
B16 = torch.bfloat16


def digits(M, C, O, R, N, cancel, seed):
    """(Y [M,C], P [N,R,C], Q [N,O,R], Wt [O,C], scale [N], ids [M]) of
    t = scale Y P_a^T,  out = Y Wt^T + t Q_a^T."""
    g = torch.Generator().manual_seed(seed)
    Y = torch.zeros((M, C))
    P, Q, Wt = torch.zeros((N, R, C)), torch.zeros((N, O, R)), torch.zeros((O, C))
    # eight triples of features, spread over the reduction: 2^16 p0, 2^8 p1, p2
    place = torch.randperm(C, generator=g)[:24].view(8, 3)
    for j in range(8):
        Y[:, place[j, 0]] = torch.randint(33, 64, (M,), generator=g).float() * 2 ** 16
        Y[:, place[j, 1]] = torch.randint(129, 256, (M,), generator=g).float() * 2 ** 8
        Y[:, place[j, 2]] = torch.randint(33, 64, (M,), generator=g).float()
    r, o = torch.arange(R), torch.arange(O)
    size = torch.where(r % 2 == 0, 1.0, -1.0) * 2.0 ** (r // 8 % 3)
    for j in range(3):
        P[:, r, place[r % 8, j]] = size
    own = o % R                     # the rank an output takes
    for a in range(N):
        Q[a, o, own] = (1.0 if a % 2 == 0 else 0.5) * torch.where(o % 3 == 0, -1.0, 1.0)
    scale = torch.tensor([1.0, 2.0] * N)[:N]    # scale times Q's size is 1 for every adapter
    if cancel:
        for j in range(2):
            Wt[o, place[own % 8, j]] = -size[own] * torch.where(o % 3 == 0, -1.0, 1.0)
    ids = torch.randint(0, N, (M,), generator=g, dtype=torch.int32)
    return [t.to(B16).to(DEV) for t in (Y, P, Q, Wt)] + [scale.to(DEV), ids.to(DEV)]


def expected(Y, P, Q, Wt, scale, ids):
    Yd, a = Y.double(), ids.long()
    t = torch.einsum("mc,mrc->mr", Yd, P.double()[a]) * scale.double()[a, None]
    return t, Yd @ Wt.double().T + torch.einsum("mr,mor->mo", t, Q.double()[a])


CASES = [  # M, C, O, R, N: widths of the parts (16, 32, 64 ranks and more), tiles of one and of several adapters
    (140, 128, 264, 8, 1), (260, 64, 520, 16, 3), (300, 200, 512, 24, 5), (256, 128, 256, 32, 1),
    (513, 72, 520, 40, 4), (260, 128, 1032, 64, 2), (150, 64, 264, 136, 3), (512, 64, 264, 256, 1),
    (300, 4096, 520, 16, 2), (300, 4096, 520, 48, 2),   # tiles cut along the reduction
    (1, 128, 264, 16, 1), (70, 64, 264, 40, 5),         # up to 128 tokens
]


@pytest.mark.parametrize("cancel", [False, True])
@pytest.mark.parametrize("dtype", [torch.float32, B16])
@pytest.mark.parametrize("M,C,O,R,N", CASES)
def test_logits_keep_every_bit_of_u(M, C, O, R, N, dtype, cancel):
    Y, P, Q, Wt, scale, ids = digits(M, C, O, R, N, cancel, M + R)
    rt, ref = expected(Y, P, Q, Wt, scale, ids)
    u, logits = guarded_empty((M, R)), guarded_empty((M, O), dtype)
    ws = guarded_empty((lmhead.lmhead_lora_workspace_bytes(M, C, O, R, N) // 256 * 256 + 256,), torch.uint8)
    lmhead.lmhead_fwd_lora(Y, Wt, P, Q, scale, ids, u, logits, ws)
    torch.cuda.synchronize()
    assert torch.equal(u.double(), rt)
    assert float(ref.abs().max()) < 2 ** 24 * 4 and torch.equal(ref.float().double(), ref)
    assert torch.equal(logits, ref.float().to(dtype))


@pytest.mark.parametrize("cancel", [False, True])
@pytest.mark.parametrize("dtype", [torch.float32, B16])
@pytest.mark.parametrize("M,C,O,R,N", CASES + [(1500, 520, 4096, 16, 2)])  # the last wave in parts
def test_dx_keeps_every_bit_of_g(M, C, O, R, N, dtype, cancel):
    Y, P, Q, Wt, scale, ids = digits(M, C, O, R, N, cancel, M + R + 1)
    rt, ref = expected(Y, P, Q, Wt, scale, ids)
    g, dX = guarded_empty((M, R)), guarded_empty((M, O), dtype)
    ws = guarded_empty((lmhead.lmhead_lora_workspace_bytes(M, O, C, R, N) // 256 * 256 + 256,), torch.uint8)
    lmhead.lmhead_bwd_dx_lora(Y, Wt.T.contiguous(), Q.transpose(1, 2).contiguous(),
                              P.transpose(1, 2).contiguous(), scale, ids, g, dX, ws)
    torch.cuda.synchronize()
    assert torch.equal(g.double(), rt)
    assert torch.equal(dX, ref.float().to(dtype))


@pytest.mark.parametrize("R", [8, 16, 24, 32, 48, 64, 136])
def test_adapter_gradients_keep_every_bit(R):
    """u and g of 23 bits, each token with a column of its own in dlogits and X: one product
    with a power of two per element of dA and dB."""
    M, N = 300, 4
    K = V = 304
    gen = torch.Generator().manual_seed(R)
    u, g = ((torch.randint(2 ** 22, 2 ** 23, (M, R), generator=gen) | 1) *
            (1 - 2 * torch.randint(0, 2, (M, R), generator=gen)) for _ in range(2))
    u, g = (u.double() * 2.0 ** -21).float().to(DEV), (g.double() * 2.0 ** -21).float().to(DEV)
    ids = torch.randint(-1, N, (M,), generator=gen, dtype=torch.int32).to(DEV)
    at = torch.arange(M, device=DEV)
    dl, X = torch.zeros((M, V), dtype=B16, device=DEV), torch.zeros((M, K), dtype=B16, device=DEV)
    dl[at, at], X[at, at + 3] = 0.5, -2.0
    dA, dB = guarded_empty((N, R, K)), guarded_empty((N, V, R))
    ws = guarded_empty((lmhead.lmhead_lora_workspace_bytes(M, K, V, R, N) // 256 * 256 + 256,), torch.uint8)
    lmhead.lmhead_bwd_lora(dl, X, u, g, ids, dA, dB, ws)
    torch.cuda.synchronize()
    rA, rB = torch.zeros((N, R, K), device=DEV), torch.zeros((N, V, R), device=DEV)
    for i in range(M):
        a = int(ids[i])
        if a >= 0:
            rA[a, :, i + 3], rB[a, i] = g[i] * -2.0, u[i] * 0.5
    assert torch.equal(dA, rA) and torch.equal(dB, rB)


LARGEST = torch.finfo(torch.float32).max   # 24 bits; rounded to nearest BF16 it would be infinite


@pytest.mark.parametrize("M", [5, 140, 300])
@pytest.mark.parametrize("R", [8, 32, 64])
def test_the_largest_u_and_g_stay_finite(M, R):
    K, V, N = 64, 264, 2
    X, W, A, B = (torch.zeros(s, dtype=B16, device=DEV) for s in ((M, K), (V, K), (N, R, K), (N, V, R)))
    X[:, 0], A[:, 3, 0], B[:, :, 3] = 1.0, 1.0, 2.0 ** -126
    scale = torch.tensor([LARGEST, -LARGEST], device=DEV)
    ids = (torch.arange(M, device=DEV) % 2).int()
    u, logits = guarded_empty((M, R)), guarded_empty((M, V))
    ws = guarded_empty((lmhead.lmhead_lora_workspace_bytes(M, K, V, R, N) // 256 * 256 + 256,), torch.uint8)
    lmhead.lmhead_fwd_lora(X, W, A, B, scale, ids, u, logits, ws)
    want = scale[ids.long()]
    torch.cuda.synchronize()
    assert torch.equal(u[:, 3], want) and not u[:, :3].any() and not u[:, 4:].any()
    assert torch.equal(logits, (want * 2.0 ** -126)[:, None].expand(M, V))
    # the gradients' split of the same u, one token per column
    dl = torch.zeros((M, V), dtype=B16, device=DEV)
    at = torch.arange(min(M, V), device=DEV)
    dl[at, at] = 2.0 ** -126
    dA, dB = guarded_empty((N, R, K)), guarded_empty((N, V, R))
    lmhead.lmhead_bwd_lora(dl, X, u, torch.zeros_like(u), ids, dA, dB, ws)
    torch.cuda.synchronize()
    ref = torch.zeros((N, V, R), device=DEV)
    ref[ids[at].long(), at, 3] = want[at] * 2.0 ** -126
    assert torch.equal(dB, ref) and not dA.any()
