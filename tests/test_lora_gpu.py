"""The LM head with low-rank adapters against the formulas in FP64.

Tolerances, per element, with S the sum of the absolute values of the terms:

  GEMM sums, FP32 output: per 768 terms (48 MMAs) the tensor cores lose at most
    2^-23 of the running sum per MMA and about four such inside one, then the
    parts are added in FP32: 2^-23 * (52 + terms / 1536) * S; dX per 512 terms (32
    MMAs): 2^-23 * (36 + terms / 1024) * S.  BF16 output: per 4096 terms (256
    MMAs): 2^-23 * (260 + terms / 8192) * S.
  row sums (u, g): the same per 128 terms (8 MMAs), parts added in FP64 or FP32,
    one rounding: 2^-23 * (12 + terms / 256) * S.
  u in the second product, above 128 tokens: for an FP32 output three BF16 parts,
    2^-24 of sum |u| |B|, for a BF16 output one, 2^-8 of it; beside u's own
    tolerance carried through B.
  gradients dA, dB: 256 terms (3 x 16 MMAs) at a time: 2^-23 * (52 + tokens / 512) * S.
  BF16 outputs: half a BF16 step (2^-9 of the value's power of two, so at most
    2^-8 of the value) beside these.

The norm of a whole FP32 product's error has a tighter bound, because the MMAs'
losses in a random sum grow like its square root: over a chunk of 48 MMAs of 16
terms they add to at most 2^-23 * (2/3) 48^1.5 * sqrt(16) of a term's size, the
chunks add in squares, and the sum itself grows as sqrt(terms): (2/3) 48 * 2^-23 =
3.8e-6 whatever the length; 4e-6 with the FP32 additions.
"""
import pytest
import torch

from lm_head_fp32_b200 import decode, lmhead, loss, synth
from helpers import guarded_empty

pytestmark = pytest.mark.gpu
DEV = "cuda"
E23 = 2.0 ** -23


def make(M, K, V, R, N, seed=0, order="random", std_a=None, none=True):
    g = torch.Generator().manual_seed(seed * 7919 + M + K + V)
    b16 = torch.bfloat16

    def nrm(*shape, std=1.0):
        return (torch.randn(shape, generator=g) * std).to(b16).to(DEV)

    X, W = nrm(M, K), nrm(V, K, std=0.02)
    A, B = nrm(N, R, K, std=std_a or K ** -0.5), nrm(N, V, R, std=0.02)
    scale = (torch.rand(N, generator=g) + 0.5).to(DEV)
    ids = torch.randint(-1 if none else 0, N, (M,), generator=g, dtype=torch.int32)
    if order == "runs":
        ids = ids.sort()[0]
    return X, W, A, B, scale, ids.to(DEV)


def workspace(M, K, V, R, N):
    return guarded_empty((lmhead.lmhead_lora_workspace_bytes(M, K, V, R, N) // 256 * 256 + 256,), torch.uint8)


def fwd(X, W, A, B, scale, ids, dtype=torch.float32, status=None):
    (M, K), V, (N, R) = X.shape, W.shape[0], A.shape[:2]
    u, logits = guarded_empty((M, R)), guarded_empty((M, V), dtype)
    u.fill_(7.0)
    lmhead.lmhead_fwd_lora(X, W, A, B, scale, ids, u, logits, workspace(M, K, V, R, N), status)
    torch.cuda.synchronize()
    return logits, u


def per_token(ids, N):
    """Each adapter that has tokens, and those."""
    for a in range(N):
        at = torch.nonzero(ids == a).view(-1)
        if at.numel():
            yield a, at


def gemm_eps(terms, dtype=torch.float32, chunk=768):
    chunk = chunk if dtype == torch.float32 else 4096
    return E23 * (chunk / 16 + 4 + terms / (2 * chunk))


def split_eps(M, dtype):
    return 2.0 ** -24 if M <= 128 or dtype == torch.float32 else 2.0 ** -8


def ref_fwd(X, W, A, B, scale, ids, dtype=torch.float32):
    """(u, its tolerance, logits, their tolerance) in FP64."""
    X, W, A, B, scale = (t.double() for t in (X, W, A, B, scale))
    M, K = X.shape
    N, R = A.shape[:2]
    out = X @ W.T
    tol = gemm_eps(K, dtype) * (X.abs() @ W.abs().T)
    u, tu = (torch.zeros((M, R), dtype=torch.float64, device=DEV) for _ in range(2))
    for a, at in per_token(ids, N):
        u[at] = scale[a] * (X[at] @ A[a].T)
        tu[at] = E23 * (12 + K / 256) * scale[a] * (X[at].abs() @ A[a].abs().T)
        ub = u[at].abs() @ B[a].abs().T
        out[at] += u[at] @ B[a].T
        tol[at] += tu[at] @ B[a].abs().T + (split_eps(M, dtype) + E23 * 56) * ub
    return u, tu, out, tol


def close(got, ref, tol, what):
    t = tol + (2.0 ** -8 * ref.abs() if got.dtype == torch.bfloat16 else 2.0 ** -24 * ref.abs())
    bad = ~((got.double() - ref).abs() <= t + 1e-30)
    assert not bad.any(), f"{what}: {int(bad.sum())} elements off, worst " \
        f"{float(((got.double() - ref).abs() / (t + 1e-30)).nan_to_num(9e9).max()):.2f} of the tolerance, " \
        f"first {torch.nonzero(bad)[:4].tolist()}"


SHAPES = [  # M, K, V, R, N
    (2, 8, 1, 8, 1), (130, 8, 9, 8, 2),
    (1, 64, 256, 8, 1), (1, 4096, 1000, 16, 3), (3, 72, 130, 8, 2), (16, 512, 300, 24, 5),
    (17, 200, 515, 16, 4), (33, 520, 1031, 32, 40), (64, 1024, 2048, 16, 64), (100, 256, 700, 40, 7),
    (128, 640, 384, 64, 3), (129, 264, 512, 16, 9), (256, 4096, 512, 8, 2), (300, 136, 255, 48, 300),
    (513, 512, 777, 128, 4), (260, 72, 1280, 256, 2), (1000, 320, 4096, 72, 6),
]


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("order", ["random", "runs"])
@pytest.mark.parametrize("M,K,V,R,N", SHAPES)
def test_forward(M, K, V, R, N, order, dtype):
    a = make(M, K, V, R, N, order=order)
    st = torch.zeros(1, dtype=torch.int32, device=DEV)
    logits, u = fwd(*a, dtype=dtype, status=st)
    ru, tu, rl, tl = ref_fwd(*a, dtype)
    close(u, ru, tu, "u")
    close(logits, rl, tl, "logits")
    assert int(st.item()) == 0


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("R", [8, 32, 64, 136])
def test_forward_tiles_of_one_adapter(R, dtype):
    """Tiles whose tokens all have one adapter take it in the shared product's sums, the
    last one with fewer tokens than columns; others beside them do not."""
    M, K, V = 1100, 264, 1030
    X, W, A, B, scale, _ = make(M, K, V, R, 3)
    ids = torch.zeros(M, dtype=torch.int32, device=DEV)
    for i, a in ((256, 1), (512, 2), (700, -1), (768, 1)):  # tiles 0, 1, 3 and 4 of one adapter
        ids[i:] = a
    logits, u = fwd(X, W, A, B, scale, ids, dtype)
    ru, tu, rl, tl = ref_fwd(X, W, A, B, scale, ids, dtype)
    close(u, ru, tu, "u")
    close(logits, rl, tl, "logits")


@pytest.mark.parametrize("M,K", [(300, 4096), (20, 4096), (256, 16384), (64, 8192)])
def test_forward_norm_of_the_error(M, K):
    a = make(M, K, 1024, 16, 4)
    logits, u = fwd(*a)
    ru, _, rl, _ = ref_fwd(*a)
    assert float((logits.double() - rl).norm() / rl.norm()) < 4e-6
    assert float((u.double() - ru).norm() / ru.norm()) < 4e-6


@pytest.mark.parametrize("M,K,V,R,N", [(1, 512, 300, 8, 1), (40, 1024, 515, 16, 5), (300, 2048, 1024, 32, 3),
                                       (200, 256, 512, 64, 9)])
def test_forward_exact_on_integers(M, K, V, R, N):
    g = torch.Generator().manual_seed(M)
    X, W = synth.int_bf16((M, K), 1, device=DEV), synth.int_bf16((V, K), 2, device=DEV)
    # A of 0 and +-1, mostly 0, so that |u| < 2^15 and its two BF16 parts hold it
    A = (torch.randint(-1, 2, (N, R, K), generator=g) * (torch.rand((N, R, K), generator=g) < 0.1)).to(torch.bfloat16).to(DEV)
    B = synth.int_bf16((N, V, R), 3, device=DEV)
    scale = torch.tensor([[1.0, 2.0, 4.0][i % 3] for i in range(N)], device=DEV)
    ids = torch.randint(-1, N, (M,), generator=g, dtype=torch.int32).to(DEV)
    logits, u = fwd(X, W, A, B, scale, ids)
    ru, _, rl, _ = ref_fwd(X, W, A, B, scale, ids)
    assert float(ru.abs().max()) < 2 ** 15
    assert torch.equal(u.double(), ru) and torch.equal(logits.double(), rl)


def pick(t, rows):
    return t[rows].double()


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("order", ["random", "runs"])
@pytest.mark.parametrize("M,K,V,R,N", [  # tiles of the logits cut along K
    (1, 4096, 129, 8, 1), (2, 4096, 4096, 16, 4), (16, 2056, 1001, 64, 20), (17, 4096, 4097, 24, 5),
    (32, 1544, 2048, 256, 3), (50, 4096, 3999, 16, 60), (64, 8192, 515, 40, 1), (128, 4096, 2000, 16, 9),
    (127, 3200, 1023, 136, 40), (200, 4096, 600, 16, 3), (300, 4096, 4099, 64, 30), (700, 8200, 1300, 8, 257),
])
def test_forward_cut_along_the_reduction(M, K, V, R, N, order, dtype):
    X, W, A, B, scale, ids = make(M, K, V, R, N, order=order)
    logits, u = fwd(X, W, A, B, scale, ids, dtype)
    ru, tu, ref, tol = ref_fwd(X, W, A, B, scale, ids, dtype)
    close(u, ru, tu, "u")
    close(logits, ref, tol, "logits")
    again, _ = fwd(X, W, A, B, scale, ids, dtype)
    assert torch.equal(logits, again)


@pytest.mark.parametrize("M", [5, 70, 300])
def test_cut_forward_keeps_bad_values_apart(M):
    X, W, A, B, scale, ids = make(M, 4096, 700, 16, 3)
    ids[::3] = 1
    one, _ = fwd(X, W, A, B, scale, ids)
    A2, B2 = A.clone(), B.clone()
    A2[1], B2[1, 5:300] = float("nan"), float("inf")
    two, _ = fwd(X, W, A2, B2, scale, ids)
    o = ids != 1
    assert torch.equal(one[o], two[o]) and torch.isnan(two[~o]).all()


@pytest.mark.parametrize("M", [5, 260])
def test_adapters_beyond_32_bit_offsets(M):
    K, V, R, N = 256, 32776, 128, 600   # B has 2.5e9 elements
    g = torch.Generator(device=DEV).manual_seed(M)
    b16 = torch.bfloat16
    X = torch.randn((M, K), generator=g, device=DEV).to(b16)
    W = (torch.randn((V, K), generator=g, device=DEV) * 0.02).to(b16)
    A = (torch.randn((N, R, K), generator=g, device=DEV) * K ** -0.5).to(b16)
    B = torch.empty((N, V, R), dtype=b16, device=DEV)
    for a in range(0, N, 50):
        B[a:a + 50] = torch.randn((50, V, R), generator=g, device=DEV).mul_(0.02)
    scale = torch.ones(N, device=DEV)
    ids = torch.full((M,), 599, dtype=torch.int32, device=DEV)
    ids[:2], ids[-1] = 598, 0
    dl = torch.randn((M, V), generator=g, device=DEV).mul_(0.01).to(b16)
    logits, u = fwd(X, W, A, B, scale, ids)
    ws = workspace(M, K, V, R, N)
    gt, dX = guarded_empty((M, R)), guarded_empty((M, K))
    lmhead.lmhead_bwd_dx_lora(dl, W, A, B, scale, ids, gt, dX, ws)
    dA = torch.empty((N, R, K), device=DEV)
    dB = torch.empty((N, V, R), device=DEV)
    lmhead.lmhead_bwd_lora(dl, X, u, gt, ids, dA, dB, ws)
    torch.cuda.synchronize()
    for a, at in per_token(ids, N):
        x, d, Aa, Ba = pick(X, at), pick(dl, at), A[a].double(), B[a].double()
        ut, gg = x @ Aa.T, d @ Ba
        tu = E23 * (12 + K / 256) * (x.abs() @ Aa.abs().T)
        tg = E23 * (12 + V / 256) * (d.abs() @ Ba.abs())
        close(u[at], ut, tu, "u")
        close(gt[at], gg, tg, "g")
        close(logits[at], x @ W.double().T + ut @ Ba.T,
              gemm_eps(K) * (x.abs() @ W.double().abs().T) + tu @ Ba.abs().T
              + (split_eps(M, torch.float32) + E23 * 56) * (ut.abs() @ Ba.abs().T), "logits")
        close(dX[at], d @ W.double() + gg @ Aa,
              gemm_eps(V, chunk=512) * (d.abs() @ W.double().abs()) + tg @ Aa.abs()
              + (split_eps(M, torch.float32) + E23 * 56) * (gg.abs() @ Aa.abs()), "dX")
        sum_tol = E23 * (52 + M / 512)
        close(dA[a], gg.T @ x, tg.T @ x.abs() + sum_tol * (gg.abs().T @ x.abs()), "dA")
        close(dB[a], d.T @ ut, d.abs().T @ tu + sum_tol * (d.abs().T @ ut.abs()), "dB")
    for a in (1, 300, 597):
        assert not dA[a].any() and not dB[a].any()


@pytest.mark.parametrize("V", [131080, 131083])
def test_logits_beyond_32_bit_offsets(V):
    M, K, R, N = 16500, 64, 8, 3       # 2.16e9 logits
    X, W, A, B, scale, ids = make(M, K, V, R, N)
    logits, u = fwd(X, W, A, B, scale, ids, torch.bfloat16)
    rows = torch.tensor([0, 1, 255, 256, 8191, 16383, 16384, 16385, M - 2, M - 1], device=DEV)
    ru, tu, ref, tol = ref_fwd(X[rows], W, A, B, scale, ids[rows], torch.bfloat16)
    # ten rows alone would take u in FP32; the whole batch takes it as one BF16 part
    for a, at in per_token(ids[rows], N):
        tol[at] += 2.0 ** -8 * (ru[at].abs() @ B[a].double().abs().T)
    close(u[rows], ru, tu, "u")
    close(logits[rows], ref, tol, "logits")


def test_adapter_order_does_not_matter_and_is_deterministic():
    X, W, A, B, scale, ids = make(300, 512, 1024, 16, 6, none=True)
    one, u1 = fwd(X, W, A, B, scale, ids)
    two, u2 = fwd(X, W, A, B, scale, ids)
    assert torch.equal(one, two) and torch.equal(u1, u2)
    perm = torch.randperm(300, generator=torch.Generator().manual_seed(4)).to(DEV)
    three, u3 = fwd(X[perm].contiguous(), W, A, B, scale, ids[perm].contiguous())
    # a token's sums do not depend on its neighbours
    assert torch.equal(one[perm], three) and torch.equal(u1[perm], u3)


@pytest.mark.parametrize("M,N,R", [(1, 3, 16), (16, 9, 16), (64, 16, 64), (128, 40, 16)])
def test_forward_is_the_same_beside_other_work(M, N, R):
    X, W, A, B, scale, ids = make(M, 4096, 9000, R, N, none=True)
    one, u1 = fwd(X, W, A, B, scale, ids)
    busy, side = torch.randn((2048, 2048), device=DEV), torch.cuda.Stream()
    for i in range(20):
        with torch.cuda.stream(side):
            for _ in range(i % 4):
                busy @ busy
        two, u2 = fwd(X, W, A, B, scale, ids)
        assert torch.equal(one, two) and torch.equal(u1, u2)
    perm = torch.randperm(M, generator=torch.Generator().manual_seed(4)).to(DEV)
    two, u2 = fwd(X[perm].contiguous(), W, A, B, scale, ids[perm].contiguous())
    assert torch.equal(one[perm], two) and torch.equal(u1[perm], u2)


@pytest.mark.parametrize("M", [5, 70, 300])
def test_bad_values_stay_with_their_adapter(M):
    X, W, A, B, scale, ids = make(M, 256, 515, 16, 3, none=True)
    ids[::4] = 1
    ids[1::4] = 0
    ref, uref = fwd(X, W, A, B, scale, ids)
    A2, B2 = A.clone(), B.clone()
    A2[1, 3, 5] = float("nan")
    B2[1, 7] = float("inf")
    B2[1, 400:] = float("nan")
    got, u = fwd(X, W, A2, B2, scale, ids)
    others = ids != 1
    assert torch.equal(got[others], ref[others]) and torch.equal(u[others], uref[others])
    assert not torch.isfinite(got[~others]).all()
    X2 = X.clone()
    X2[2] = float("nan")
    got, _ = fwd(X2, W, A, B, scale, ids)
    keep = torch.arange(M, device=DEV) != 2
    assert torch.equal(got[keep], ref[keep])


def test_u_beyond_bf16_keeps_its_sign():
    X, W, A, B, scale, ids = make(4, 64, 300, 8, 1, none=False)
    scale[:] = 3e38
    X[:] = X.abs()
    A[:] = 4.0
    B[:] = B.abs() + 0.01
    logits, u = fwd(X, W, A, B, scale, ids)
    assert torch.isinf(u).all() and (logits == float("inf")).all()


def test_ids_out_of_range_and_none():
    X, W, A, B, scale, ids = make(70, 128, 512, 8, 3)
    ids[:] = -1
    st = torch.zeros(1, dtype=torch.int32, device=DEV)
    base, u = fwd(X, W, A, B, scale, ids, status=st)
    assert int(st.item()) == 0 and not u.any()
    close(base, X.double() @ W.double().T, gemm_eps(128) * (X.double().abs() @ W.double().abs().T), "base")
    ids[3], ids[69] = 3, -2
    got, u = fwd(X, W, A, B, scale, ids, status=st)
    assert int(st.item()) == lmhead.DEV_BAD_ADAPTER and torch.equal(got, base) and not u.any()


def test_logits_off_alignment_are_the_same():
    X, W, A, B, scale, ids = make(70, 256, 516, 16, 4)
    ref, _ = fwd(X, W, A, B, scale, ids)
    buf = torch.full((70 * 516 + 8,), 7.0, device=DEV)
    out = buf[3:3 + 70 * 516].view(70, 516)
    lmhead.lmhead_fwd_lora(X, W, A, B, scale, ids, torch.empty((70, 16), device=DEV), out,
                           workspace(70, 256, 516, 16, 4))
    assert torch.equal(out, ref) and (buf[:3] == 7).all() and (buf[3 + 70 * 516:] == 7).all()


# ------------------------------------------------------------------ backward

def bwd(dl, X, W, A, B, scale, ids, u, dtype=torch.float32, status=None):
    (M, K), V, (N, R) = X.shape, W.shape[0], A.shape[:2]
    g, dX = guarded_empty((M, R)), guarded_empty((M, K), dtype)
    dA, dB = guarded_empty((N, R, K)), guarded_empty((N, V, R))
    ws = workspace(M, K, V, R, N)
    lmhead.lmhead_bwd_dx_lora(dl, W, A, B, scale, ids, g, dX, ws, status)
    lmhead.lmhead_bwd_lora(dl, X, u, g, ids, dA, dB, ws, status)
    torch.cuda.synchronize()
    return g, dX, dA, dB


def check_bwd(M, K, V, R, N, order, dtype, seed=0):
    X, W, A, B, scale, ids = make(M, K, V, R, N, seed, order)
    gen = torch.Generator().manual_seed(V)
    dl = (torch.randn((M, V), generator=gen) * 1e-3).to(torch.bfloat16).to(DEV)
    u = torch.randn((M, R), generator=gen).to(DEV)
    st = torch.zeros(1, dtype=torch.int32, device=DEV)
    g, dX, dA, dB = bwd(dl, X, W, A, B, scale, ids, u, dtype, st)
    assert int(st.item()) == 0
    Xd, Wd, Ad, Bd, sd, dd, ud = (t.double() for t in (X, W, A, B, scale, dl, u))
    rg, tg = (torch.zeros((M, R), dtype=torch.float64, device=DEV) for _ in range(2))
    rX, tX = dd @ Wd, gemm_eps(V, dtype, 512) * (dd.abs() @ Wd.abs())
    for a in range(N):
        at = torch.nonzero(ids == a).view(-1)
        rg[at] = sd[a] * (dd[at] @ Bd[a])
        tg[at] = E23 * (12 + V / 256) * sd[a] * (dd[at].abs() @ Bd[a].abs())
        rX[at] += rg[at] @ Ad[a]
        tX[at] += tg[at] @ Ad[a].abs() + (split_eps(M, dtype) + E23 * 56) * (rg[at].abs() @ Ad[a].abs())
        c = E23 * (52 + at.numel() / 512)
        gf = g[at].double()  # as the call was given it
        close(dA[a], gf.T @ Xd[at], c * (gf.abs().T @ Xd[at].abs()), f"dA[{a}]")
        close(dB[a], dd[at].T @ ud[at], c * (dd[at].abs().T @ ud[at].abs()), f"dB[{a}]")
        if not at.numel():
            assert not dA[a].any() and not dB[a].any()
    close(g, rg, tg, "g")
    close(dX, rX, tX, "dX")


@pytest.mark.parametrize("order", ["random", "runs"])
@pytest.mark.parametrize("M,K,V,R,N", [
    (2, 8, 8, 8, 1), (130, 8, 16, 8, 2),
    (1, 64, 256, 8, 1), (3, 72, 136, 8, 2), (16, 512, 304, 24, 5), (33, 520, 1032, 32, 40),
    (64, 1024, 2048, 16, 64), (129, 264, 512, 16, 9), (300, 136, 256, 48, 300), (513, 512, 776, 128, 4),
    (260, 72, 1280, 256, 2), (1000, 320, 4096, 72, 6), (70, 128, 20000, 64, 3), (1100, 256, 1024, 16, 1),
    (530, 64, 65536, 24, 7),  # the rows taken adapter by adapter
    (1500, 4096, 512, 16, 2),  # several tiles per CTA, tiles of one adapter, the last wave in halves
    (2000, 4096, 520, 40, 3),  # the last wave with three short parts per idle unit
])
def test_backward(M, K, V, R, N, order):
    check_bwd(M, K, V, R, N, order, torch.bfloat16 if M % 2 else torch.float32)


@pytest.mark.parametrize("order", ["random", "runs"])
@pytest.mark.parametrize("M,K,V,R,N", [  # every tile of dX cut along the vocabulary
    (1, 8, 4096, 8, 1), (16, 512, 2056, 8, 3), (60, 792, 9000, 16, 4), (37, 136, 40000, 24, 40),
    (64, 2048, 8192, 256, 5), (100, 1024, 16392, 48, 90), (128, 256, 5000, 16, 2), (127, 4096, 6000, 8, 1),
    (200, 200, 9000, 40, 6), (300, 1032, 12296, 32, 7), (513, 256, 33000, 64, 3), (257, 3000, 4104, 16, 257),
])
def test_backward_cut_along_the_vocabulary(M, K, V, R, N, order):
    check_bwd(M, K, V, R, N, order, torch.bfloat16 if V % 16 else torch.float32)


@pytest.mark.parametrize("M", [40, 120, 300])
def test_cut_backward_is_deterministic_and_keeps_bad_values_apart(M):
    V = 6000
    X, W, A, B, scale, ids = make(M, 512, V, 16, 3)
    ids[::3] = 1
    gen = torch.Generator().manual_seed(4)
    dl = torch.randn((M, V), generator=gen).to(torch.bfloat16).to(DEV)
    u = torch.randn((M, 16), generator=gen).to(DEV)
    ref = bwd(dl, X, W, A, B, scale, ids, u)
    for _ in range(20):
        for p, q in zip(ref, bwd(dl, X, W, A, B, scale, ids, u)):
            assert torch.equal(p, q)
    A2, B2 = A.clone(), B.clone()
    A2[1], B2[1, 100:200] = float("nan"), float("inf")
    got = bwd(dl, X, W, A2, B2, scale, ids, u)
    o = ids != 1
    assert torch.equal(got[0][o], ref[0][o]) and torch.equal(got[1][o], ref[1][o])
    assert torch.isnan(got[1][~o]).all()


def test_backward_long_reduction_norm():
    X, W, A, B, scale, ids = make(256, 256, 65536, 16, 4)
    dl = torch.randn((256, 65536), generator=torch.Generator().manual_seed(1)).to(torch.bfloat16).to(DEV)
    u = torch.randn((256, 16), generator=torch.Generator().manual_seed(2)).to(DEV)
    g, dX, dA, dB = bwd(dl, X, W, A, B, scale, ids, u)
    rX = dl.double() @ W.double()
    rg = torch.zeros((256, 16), dtype=torch.float64, device=DEV)
    for a in range(4):
        at = torch.nonzero(ids == a).view(-1)
        rg[at] = scale[a].double() * (dl[at].double() @ B[a].double())
        rX[at] += rg[at] @ A[a].double()
    assert float((dX.double() - rX).norm() / rX.norm()) < 4e-6
    assert float((g.double() - rg).norm() / rg.norm()) < 4e-6


def test_backward_bad_values_stay_with_their_adapter():
    X, W, A, B, scale, ids = make(150, 128, 512, 16, 3)
    ids[::3] = 1
    gen = torch.Generator().manual_seed(3)
    dl = torch.randn((150, 512), generator=gen).to(torch.bfloat16).to(DEV)
    u = torch.randn((150, 16), generator=gen).to(DEV)
    ref = bwd(dl, X, W, A, B, scale, ids, u)
    A2, B2, u2 = A.clone(), B.clone(), u.clone()
    A2[1], B2[1, 100:200], u2[0] = float("nan"), float("inf"), float("nan")
    got = bwd(dl, X, W, A2, B2, scale, ids, u2)
    o = ids != 1
    assert torch.equal(got[0][o], ref[0][o]) and torch.equal(got[1][o], ref[1][o])
    for a in (0, 2):
        assert torch.equal(got[2][a], ref[2][a]) and torch.equal(got[3][a], ref[3][a])
    assert torch.isnan(got[3][1]).any()


# ------------------------------------------------------------------ the loss

def loss_inputs(M=150, K=128, V=1000, R=16, N=3, seed=5):
    X, W, A, B, scale, ids = make(M, K, V, R, N, seed)
    t = synth.targets(M, V, 0.1, 9).to(DEV)
    return X, W, A, B, scale, ids, t


def test_loss_gradients_match_the_formula():
    X, W, A, B, scale, ids, t = loss_inputs()
    leaves = [p.clone().requires_grad_() for p in (X, W, A, B)]
    out = loss.lm_head_lora_cross_entropy(*leaves, scale, ids, t)
    n = int((t != -100).sum())
    (out.sum() / n).backward()
    d = [p.double().requires_grad_() for p in (X, W, A, B)]
    idl = ids.long().clamp(min=0)
    on = (ids >= 0).double() * scale.double()[idl]
    un = torch.einsum("mk,mrk->mr", d[0], d[2][idl]) * on[:, None]
    lg = d[0] @ d[1].T + torch.einsum("mr,mvr->mv", un, d[3][idl])
    ref = torch.nn.functional.cross_entropy(lg, t, reduction="none", ignore_index=-100)
    (ref.sum() / n).backward()
    assert ((out.double() - ref).abs() <= 1e-5 * ref.abs() + 1e-5).all()
    # each gradient is a product with BF16 dlogits (2^-8 of each, random in sign)
    # and is itself rounded to BF16
    for got, want in zip(leaves, d):
        assert float((got.grad.double() - want.grad).norm() / want.grad.norm()) < 2.0 ** -8


@pytest.mark.parametrize("which", [2, 3])
def test_loss_gradient_against_differences(which):
    """The derivative along a direction that moves each weight by 2^-8 (A and B are
    multiples of 2^-8 of at most 2^-3, so that weight +- step is exact in BF16): central
    differences of the FP32 loss.  The loss of a token is good to 1e-5, there are 150,
    and the direction is the gradient's sign, so that the slope is large."""
    X, W, A, B, scale, ids, t = loss_inputs()
    gen = torch.Generator().manual_seed(8)

    def grid(shape):
        return (torch.randint(-32, 33, shape, generator=gen) / 256).to(torch.bfloat16).to(DEV)

    A, B = grid(A.shape), grid(B.shape)
    args = [X, W, A.requires_grad_(), B.requires_grad_()]
    loss.lm_head_lora_cross_entropy(*args, scale, ids, t).double().sum().backward()
    grad = args[which].grad.double()
    h = 2.0 ** -8
    step = torch.sign(grad) * h
    step[grad.abs() < grad.abs().max() * 0.05] = 0

    def at(sign):
        p = [q.detach() for q in args]
        moved = (p[which].double() + sign * step)
        assert torch.equal(moved.to(torch.bfloat16).double(), moved)
        p[which] = moved.to(torch.bfloat16)
        return float(loss.lm_head_lora_cross_entropy(*p, scale, ids, t).double().sum())

    slope = float((grad * step).sum())
    # the quadratic term cancels; the cubic one is below a twentieth at this step
    assert abs((at(1) - at(-1)) / 2 - slope) <= 0.05 * abs(slope)


def test_loss_captured_while_an_eager_graph_lives():
    X, W, A, B, scale, ids, t = loss_inputs()
    A.requires_grad_(), B.requires_grad_()
    eager = loss.lm_head_lora_cross_entropy(X, W, A, B, scale, ids, t).sum()
    ga, gb = torch.autograd.grad(eager, (A, B), retain_graph=True)
    a2, b2 = A.detach().clone().requires_grad_(), B.detach().clone().requires_grad_()
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        out = loss.lm_head_lora_cross_entropy(X, W, a2, b2, scale, ids, t, status=status).sum()
        torch.autograd.grad(out, (a2, b2))
    torch.cuda.current_stream().wait_stream(s)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = loss.lm_head_lora_cross_entropy(X, W, a2, b2, scale, ids, t, status=status).sum()
        da, db = torch.autograd.grad(out, (a2, b2))
    for _ in range(2):
        graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, eager.detach()) and torch.equal(da, ga) and torch.equal(db, gb)


# ------------------------------------------------------------------ together

@pytest.mark.parametrize("lora", [False, True])
def test_decode_steps(lora):
    """Beam search over a toy model (the state of a beam is its hidden vector and its
    history): every step's choice and states against a restatement in FP64."""
    E, Wd, K, V, R, N, eos = 3, 4, 64, 1003, 8, 2, 5
    X, W, A, B, scale, _ = make(E * Wd, K, V, R, N, 3)
    W = (W.float() * 8).to(torch.bfloat16)
    emb = make(V, K, 8, 8, 1, 4)[0]
    ids = torch.tensor([0, -1, 1], dtype=torch.int32, device=DEV).repeat_interleave(Wd)
    dec = decode.BeamDecoder(W, E, Wd, eos, *((A, B, scale) if lora else ()))
    hidden = X.view(E, Wd, K).clone()
    hist = torch.zeros((E, Wd, 6), dtype=torch.int64, device=DEV)
    rh, rhist = hidden.double(), hist.clone()
    rs = torch.full((E, Wd), float("-inf"), dtype=torch.float64, device=DEV)
    rs[:, 0] = 0
    for t in range(5):
        x = hidden.reshape(-1, K)
        tok, par, sc = dec.step(x, [hist], adapter=ids if lora else None)
        lmhead.beam_reorder(hidden, par)
        # the restatement, from the same hidden states
        lg = rh.reshape(-1, K) @ W.double().T
        if lora:
            for a in range(N):
                at = torch.nonzero(ids == a).view(-1)
                lg[at] += scale[a].double() * (rh.reshape(-1, K)[at] @ A[a].double().T) @ B[a].double().T
        tot = (lg.log_softmax(1).view(E, Wd, V) + rs[:, :, None]).view(E, -1)
        best = tot.sort(dim=1, descending=True, stable=True)
        for e in range(E):
            on = [int(i) for i in best.indices[e, :2 * Wd] if int(i) % V != eos][:Wd]
            assert [i // V for i in on] == par[e].tolist() and [i % V for i in on] == tok[e].tolist()
            rs[e] = tot[e, on]
            rh[e], rhist[e] = rh[e, [i // V for i in on]], rhist[e, [i // V for i in on]]
        assert ((sc.double() - rs).abs() <= 1e-4 * (t + 1)).all()
        assert torch.equal(hist, rhist) and torch.equal(hidden.double(), rh)
        hist[:, :, t], rhist[:, :, t] = tok, tok
        hidden = (hidden.float() * 0.5 + emb[tok].float()).to(torch.bfloat16).contiguous()
        rh = hidden.double()
        rs = sc.double()
    assert int(dec.status.item()) == 0


def test_decode_step_captured():
    E, Wd, K, V, R, N = 2, 3, 128, 2000, 16, 3
    X, W, A, B, scale, ids = make(E * Wd, K, V, R, N, 6)
    hist = torch.arange(E * Wd, device=DEV).view(E, Wd, 1).contiguous()
    dec = decode.BeamDecoder(W, E, Wd, 1, A, B, scale)
    ref = decode.BeamDecoder(W, E, Wd, 1, A, B, scale)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        dec.step(X, [hist], adapter=ids)
    dec.reset()
    hist.copy_(torch.arange(E * Wd, device=DEV).view(E, Wd, 1))
    rhist = hist.clone()
    for t in range(3):
        X.copy_(make(E * Wd, K, V, R, N, 10 + t)[0])
        g.replay()
        ref.step(X, [rhist], adapter=ids)
        torch.cuda.synchronize()
        for f in ("tokens", "parents", "scores", "cand_token"):
            assert torch.equal(getattr(dec, f), getattr(ref, f)), f
        assert torch.equal(hist, rhist)


def test_two_streams_at_once():
    """Two forwards with workspaces of their own, on two streams at the same time."""
    a, b = make(200, 512, 4096, 16, 4, 1), make(64, 512, 4096, 16, 4, 2)
    ra, rb = fwd(*a), fwd(*b)
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    for _ in range(3):
        with torch.cuda.stream(s1):
            (M, K), (V, _) = a[0].shape, a[1].shape
            la, ua, wa = torch.empty((M, V), device=DEV), torch.empty((M, 16), device=DEV), workspace(M, K, V, 16, 4)
            lmhead.lmhead_fwd_lora(*a, ua, la, wa)
        with torch.cuda.stream(s2):
            (M, K), (V, _) = b[0].shape, b[1].shape
            lb, ub, wb = torch.empty((M, V), device=DEV), torch.empty((M, 16), device=DEV), workspace(M, K, V, 16, 4)
            lmhead.lmhead_fwd_lora(*b, ub, lb, wb)
        torch.cuda.synchronize()
        assert torch.equal(la, ra[0]) and torch.equal(lb, rb[0]) and torch.equal(ua, ra[1])
