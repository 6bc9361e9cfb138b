"""beam_select and beam_reorder against plain FP64 / index restatements.

Tolerance of a score: rounding the FP64 total to FP32 costs 2^-24 |total|.  lse
is the log of a sum of positive terms, each off by at most 2^-22 (the base-2
exponential) and 2^-24 |t| for its rounded argument t (terms that matter have
|t| < 16), summed in FP32 over at most 10 additions (10 * 2^-24): below 2e-6
relative, which is 2e-6 absolute in the log.
"""
import pytest
import torch

from lm_head_fp32_b200 import lmhead
from helpers import guarded_empty, guarded_full

pytestmark = pytest.mark.gpu
DEV = "cuda"
NEG = float("-inf")


def plain_select(logits, scores, C, eos, done=None):
    """The definition in FP64 on the CPU, with the documented fill of empty places."""
    x = logits.double().cpu()
    x = torch.where(x < 1e38, x, torch.full_like(x, NEG))
    s = scores.double().cpu()
    s = torch.where(s < float("inf"), s, torch.full_like(s, NEG))
    N, W, V = x.shape
    m = x.amax(2, keepdim=True)
    m0 = torch.where(m > NEG, m, torch.zeros_like(m))
    lse = (x - m0).exp().sum(2, keepdim=True).log() + m0
    total = torch.where(x > NEG, s[:, :, None] + x - lse, x)
    # equal totals: the lower beam, the higher logit, the lower token
    by_logit = x.sort(dim=2, descending=True, stable=True)[1]
    val, at = total.gather(2, by_logit).view(N, W * V).sort(dim=1, descending=True, stable=True)
    at = (at // V) * V + by_logit.view(N, W * V).gather(1, at)
    cs = torch.full((N, C), NEG, dtype=torch.float64)
    cb, ct = torch.full((N, C), -1), torch.full((N, C), -1)
    ns, nb = torch.full((N, W), NEG, dtype=torch.float64), torch.arange(W).repeat(N, 1)
    nt = torch.full((N, W), max(eos, 0))
    for n in range(N):
        if done is not None and done[n]:
            ns[n] = scores[n].double().cpu()
            continue
        k = min(C, int((val[n] > NEG).sum()))
        cs[n, :k], cb[n, :k], ct[n, :k] = val[n, :k], at[n, :k] // V, at[n, :k] % V
        on = [i for i in range(k) if int(ct[n, i]) != eos][:W]
        for j, i in enumerate(on):
            ns[n, j], nb[n, j], nt[n, j] = cs[n, i], cb[n, i], ct[n, i]
    return cs, cb, ct, ns, nb, nt


def run_select(logits, scores, C, eos=-1, done=None, nxt=True, status=None):
    N, W, V = logits.shape
    out = [guarded_empty((N, C)), guarded_empty((N, C), torch.int32), guarded_empty((N, C), torch.int64)]
    out += [guarded_empty((N, W)), guarded_empty((N, W), torch.int32),
            guarded_empty((N, W), torch.int64)] if nxt else [None] * 3
    ws = guarded_empty((lmhead.beam_select_workspace_bytes(N, W, V, C),), torch.uint8)
    lmhead.beam_select(logits, scores, *out, ws, eos=eos, done=done, status=status)
    torch.cuda.synchronize()
    return out


def check(logits, scores, C, eos=-1, done=None):
    st = torch.zeros(1, dtype=torch.int32, device=DEV)
    got = run_select(logits, scores, C, eos, done, status=st)
    ref = plain_select(logits, scores, C, eos, None if done is None else done.cpu())
    for i in (1, 2, 4, 5):
        assert torch.equal(got[i].cpu().long(), ref[i]), i
    for i in (0, 3):
        g, r = got[i].cpu().double(), ref[i]
        fin = torch.isfinite(r)
        assert torch.equal(torch.isfinite(g), fin) and torch.equal(g[~fin], r[~fin])
        assert ((g - r).abs()[fin] <= 2.0 ** -24 * r.abs()[fin] + 2e-6).all()
    return got, int(st.item())


def data(N, W, V, seed, dtype=torch.float32, std=2.5):
    g = torch.Generator().manual_seed(seed)
    x = (torch.randn((N, W, V), generator=g) * std).to(dtype)
    s = -torch.rand((N, W), generator=g) * 6
    return x.to(DEV), s.to(DEV)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("N,W,V,C,eos", [
    (1, 1, 1, 1, -1), (1, 1, 2, 2, 1), (3, 2, 5, 4, 0), (2, 4, 31, 8, 3), (1, 4, 1000, 8, 2),
    (2, 3, 8191, 6, 2), (2, 3, 8192, 6, 8191), (2, 3, 8193, 6, 8192), (1, 5, 32771, 10, 2),
    (1, 2, 128256, 4, 2), (2, 16, 3001, 32, 7), (1, 64, 9000, 128, 5), (5, 7, 300, 7, -1),
    (1, 1, 500, 128, 4), (70, 1, 77, 2, 1),
])
def test_select(N, W, V, C, eos, dtype):
    x, s = data(N, W, V, 11 + V, dtype)
    if dtype == torch.bfloat16:
        # distinct totals across beams, so that FP64 reference and kernel cannot
        # differ over a gap smaller than lse's tolerance; ties inside a row stay
        s = (s * 0.7 + torch.arange(W, device=DEV) * 0.0137)
    assert check(x, s, C, eos)[1] == 0


def test_select_without_next():
    x, s = data(2, 3, 900, 5)
    got = run_select(x, s, 2, nxt=False)
    ref = plain_select(x, s, 2, -1)
    assert torch.equal(got[1].cpu().long(), ref[1]) and torch.equal(got[2].cpu().long(), ref[2])


@pytest.mark.parametrize("V", [6, 8192, 20001])
def test_equal_logits_fall_by_place(V):
    # every logit equal: more values at the threshold than the block's buffer
    x = torch.full((2, 3, V), 1.25, device=DEV)
    check(x, torch.zeros(2, 3, device=DEV), 6, eos=1)


def test_equal_logits_in_long_parts():
    # parts of several batches: more sixteens at the threshold than a warp can list
    N, V, C = 64, 300001, 6
    got = run_select(torch.full((N, 1, V), -0.5, device=DEV), torch.zeros(N, 1, device=DEV), C)
    lse = -0.5 + torch.tensor(float(V)).double().log()
    assert torch.equal(got[2].cpu(), torch.arange(C).repeat(N, 1)) and not got[1].any()
    assert ((got[0].cpu().double() - (-0.5 - lse)).abs() <= 2.0 ** -24 * 13 + 2e-6).all()


def test_few_tokens_allowed_in_long_parts():
    N, V, C = 64, 300001, 4
    x = torch.full((N, 1, V), NEG, device=DEV)
    at = torch.tensor([3, 70000, 299999], device=DEV) + torch.arange(N, device=DEV)[:, None] % 2
    x.scatter_(2, at[:, None], torch.tensor([1.0, 3.0, 2.0], device=DEV).expand(N, 1, 3).contiguous())
    got = run_select(x, torch.zeros(N, 1, device=DEV), C)
    ref = torch.tensor([3.0, 2.0, 1.0]).double().log_softmax(0)
    for n in range(N):
        assert got[2][n].tolist() == [int(at[n, 1]), int(at[n, 2]), int(at[n, 0]), -1]
        assert ((got[0][n, :3].cpu().double() - ref).abs() <= 2.0 ** -24 * 3 + 2e-6).all()
        assert got[0][n, 3].item() == NEG


@pytest.mark.parametrize("V", [4001, 32771])
def test_equal_beams_fall_by_beam(V):
    x, _ = data(2, 1, V, 3)
    x = x.expand(2, 4, V).contiguous()
    got, _ = check(x, torch.full((2, 4), -2.5, device=DEV), 8, eos=2)
    assert got[1][0, :4].tolist() == [0, 1, 2, 3]  # the best token, beam by beam


def test_first_step_and_dead_beams():
    x, s = data(3, 4, 9001, 8)
    s[:, 1:] = NEG           # one beam to begin with
    x[1, 1:] = float("nan")  # rows of dead beams are not read
    assert check(x, s, 8, eos=2)[1] == 0
    s[2] = NEG               # no beam at all
    check(x, s, 8, eos=2)


def test_masked_tokens():
    x, s = data(2, 3, 20000, 9)
    keep = torch.zeros(20000, dtype=torch.bool, device=DEV)
    keep[[5, 9000, 9001, 19999]] = True
    x[:, :, ~keep] = NEG
    x[1, 0] = NEG            # one beam with nothing allowed
    check(x, s, 6, eos=9000)
    x[:, :, 6:] = NEG        # fewer continuations than candidates
    check(x, s, 6, eos=5)


@pytest.mark.parametrize("fill", [float("nan"), float("inf"), 3e38])
def test_bad_logits_are_left_out_and_told(fill):
    x, s = data(2, 2, 8300, 10)
    x[0, 1, 7] = fill
    x[1, 0, 8299] = fill
    assert check(x, s, 4, eos=2)[1] == lmhead.DEV_BAD_LOGIT


def test_bad_scores_are_left_out_and_told():
    x, s = data(2, 2, 300, 12)
    s[0, 0], s[1, 1] = float("nan"), float("inf")
    assert check(x, s, 4, eos=2)[1] == lmhead.DEV_BAD_LOGIT


def test_done_entries_keep_their_beams():
    x, s = data(3, 2, 5000, 13)
    x[1] = float("nan")
    done = torch.tensor([0, 1, 0], dtype=torch.int32, device=DEV)
    got, st = check(x, s, 4, eos=2, done=done)
    assert st == 0 and got[4][1].tolist() == [0, 1] and got[2][1].tolist() == [-1] * 4


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("shift", [1, 2, 3, 5])
def test_rows_off_alignment(dtype, shift):
    x, s = data(2, 3, 8205, 14)
    buf = torch.full((x.numel() + 16,), float("nan"), device=DEV, dtype=dtype)
    y = buf[shift:shift + x.numel()].view(x.shape)
    y.copy_(x)
    s = s + torch.arange(3, device=DEV) * 0.0137
    assert check(y, s, 6, eos=2)[1] == 0


@pytest.mark.parametrize("kind", ["ascending", "descending", "large", "peaked"])
def test_shapes_of_rows(kind):
    x, s = data(1, 3, 30000, 15)
    if kind == "ascending":
        x = x.sort(2)[0]
    elif kind == "descending":
        x = x.sort(2, descending=True)[0]
    elif kind == "large":
        x = x * 4000          # logits of 1e4: lse keeps its last places
    else:
        x[:, :, 17] += 80
    ref = plain_select(x, s, 6, 2)
    got = run_select(x, s, 6, 2)
    for i in (1, 2, 4, 5):
        assert torch.equal(got[i].cpu().long(), ref[i])
    # a logit of 1e4 enters lse exactly (its product with log2 e is rounded at the
    # size of the difference to the maximum), so the bound is the usual one
    assert ((got[0].cpu().double() - ref[0]).abs() <= 2.0 ** -24 * ref[0].abs() + 2e-6).all()


LOWEST = torch.finfo(torch.float32).min


def far_rows(kind, dtype):
    """Rows whose largest logit is far from zero, or that mask with such logits."""
    V = 20001
    x, s = data(2, 3, V, 21, dtype)
    low = float(torch.finfo(dtype).min)
    if kind == "lowest":          # nothing but masked tokens: all equally likely
        x[:] = low
    elif kind == "one row lowest":
        x[0, 1] = low
        x[1, 2, 1:] = low
    elif kind == "parts lowest":  # whole parts of a row, and the first
        x[:, :, :13000] = low
    elif kind == "few and lowest":
        x, s = x[:, :1].contiguous(), s[:, :1].contiguous()
        keep = torch.zeros(V, dtype=torch.bool, device=DEV)
        keep[[4097, 9000, 20000]] = True
        x[:, :, ~keep] = low
    elif kind == "-1e10":
        x[0] = -1e10
        x[1, :, :19000] = -1e10
    elif kind == "1e10":
        x = (x.float() * 4e9).to(dtype)
    elif kind == "1e37":
        x = (x.float() * 1e36).to(dtype)
    elif kind == "lowest and -inf":
        x[:, :, ::2] = NEG
        x[:, :, 1::2] = low
    elif kind == "lowest score":
        s[:] = LOWEST
        s[1, 1] = -2.0
    else:                         # about where the sums change their reference
        c = {"-2^29": -1.0, "2^29": 1.0}[kind] * 2.0 ** 29
        g = torch.Generator().manual_seed(22)
        x = (c + 32.0 * torch.randint(-3, 4, x.shape, generator=g).double()).to(dtype).to(DEV)
    return x, s


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("kind", ["lowest", "one row lowest", "parts lowest", "few and lowest", "-1e10", "1e10",
                                  "1e37", "lowest and -inf", "lowest score", "-2^29", "2^29"])
def test_rows_far_from_zero(kind, dtype):
    x, s = far_rows(kind, dtype)
    # the softmax does not change when the row is shifted by its maximum, exact in
    # FP64 where it matters; without it x - lse would lose the logarithm of the sum
    m = x.double().amax(2, keepdim=True)
    C = 6
    ref = plain_select(x.double() - torch.where(m > NEG, m, torch.zeros_like(m)), s, C, 2)
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    got = run_select(x, s, C, 2, status=status)
    assert int(status.item()) == 0
    for i in (1, 2, 4, 5):
        assert torch.equal(got[i].cpu().long(), ref[i]), i
    for i in (0, 3):
        g, r = got[i].cpu().double(), ref[i]
        fin = torch.isfinite(r)
        assert torch.equal(torch.isfinite(g), fin)
        # near 2^29 the exponent's argument reaches 64: two roundings of 2^-24 * 64,
        # times ln 2, in place of those of the usual bound
        assert ((g - r).abs()[fin] <= 2.0 ** -24 * r.abs()[fin] + 2e-6 + 2 * 64 * 2.0 ** -24 * 0.7).all()


def test_zeros_of_both_signs_are_equal():
    x = torch.zeros((1, 2, 9000), device=DEV)
    x[:, :, :4] = -0.0
    x[:, 0, 5::3] = -1.0
    s = torch.tensor([[-1.0, -1.25]], device=DEV)
    check(x, s, 12, eos=1)


def test_totals_below_the_range_are_no_candidates():
    x, s = data(1, 2, 300, 23)
    x[:, :, 3:] = LOWEST
    s[:] = LOWEST
    got = run_select(x, s, 8, 2)
    # 2 x 3 continuations at the lowest value; the others would be at twice that
    assert torch.isfinite(got[0][0, :6]).all() and (got[0][0, 6:] == NEG).all()
    # their totals are equal in FP64: by beam, then by logit
    order = x[0, :, :3].argsort(1, descending=True).flatten().tolist()
    assert got[1][0].tolist() == [0, 0, 0, 1, 1, 1, -1, -1] and got[2][0].tolist() == order + [-1, -1]


def test_logits_beyond_32_bit_offsets():
    N, W, V, C = 2200, 8, 128001, 16     # 2.25e9 logits
    g = torch.Generator(device=DEV).manual_seed(24)
    x = torch.empty((N, W, V), dtype=torch.bfloat16, device=DEV)
    for n in range(0, N, 100):
        x[n:n + 100] = torch.randn((100, W, V), generator=g, device=DEV).mul_(2.5)
    s = -torch.rand((N, W), generator=g, device=DEV) * 6
    got = run_select(x, s, C, 2)
    at = [0, 1, 2047, 2048, 2097, 2098, N - 1]
    ref = plain_select(x[at], s[at], C, 2)
    for i in (1, 2, 4, 5):
        assert torch.equal(got[i][at].cpu().long(), ref[i]), i
    for i in (0, 3):
        assert ((got[i][at].cpu().double() - ref[i]).abs() <= 2.0 ** -24 * ref[i].abs() + 2e-6).all()


def test_select_twice_the_same_and_on_a_stream():
    x, s = data(4, 4, 40000, 16)
    a = run_select(x, s, 8, 2)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        b = run_select(x, s, 8, 2)
    for p, q in zip(a, b):
        assert torch.equal(p, q)


# ------------------------------------------------------------------ reorder

def plain_reorder(t, parents, e):
    N, W = parents.shape
    out = t.clone()
    for n in range(N):
        for w in range(W):
            out.select(e, n).select(e, w).copy_(t.select(e, n).select(e, int(parents[n, w])))
    return out


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.int64, torch.uint8])
@pytest.mark.parametrize("N,W,e,shape", [
    (1, 1, 0, (1, 1, 9)), (2, 3, 0, (2, 3)), (3, 4, 0, (3, 4, 33)), (2, 4, 1, (3, 2, 4, 2, 17, 5)),
    (2, 8, 0, (2, 8, 3, 64)), (1, 16, 0, (1, 16, 40)), (2, 32, 0, (2, 32, 24)), (1, 64, 0, (1, 64, 1000)),
    (2, 5, 2, (2, 3, 2, 5, 4, 16)),
])
def test_reorder(N, W, e, shape, dtype):
    g = torch.Generator().manual_seed(W * 31 + N)
    t0 = torch.randint(0, 200, shape, generator=g).to(dtype)
    par = torch.randint(0, W, (N, W), generator=g, dtype=torch.int32)
    for p in (par, torch.arange(W, dtype=torch.int32).repeat(N, 1),
              torch.arange(W, dtype=torch.int32).flip(0).repeat(N, 1),
              torch.zeros((N, W), dtype=torch.int32)):
        states = [guarded_empty(shape, dtype) for _ in range(3)]
        for i, s in enumerate(states):
            s.copy_((t0.long() + i).to(dtype))
        st = torch.zeros(1, dtype=torch.int32, device=DEV)
        lmhead.beam_reorder(states, p.to(DEV), entry_dim=e, status=st)
        for i, s in enumerate(states):
            assert torch.equal(s.cpu(), plain_reorder((t0.long() + i).to(dtype), p, e))
        assert int(st.item()) == 0


def test_reorder_beyond_32_bit_offsets():
    L, N, W, H, S, D = 2, 16, 4, 8, 20000, 128   # 5.2 GB, and the filled part of as much
    g = torch.Generator(device=DEV).manual_seed(25)
    parents = torch.randint(0, W, (N, W), generator=g, device=DEV, dtype=torch.int32)
    t = torch.randint(0, 256, (L, N, W, H, S, 2 * D), generator=g, device=DEV, dtype=torch.uint8)
    view = t[:, :, :, :, :19999]
    ref = plain_reorder(view, parents, 1)
    lmhead.beam_reorder(view, parents, 1)
    torch.cuda.synchronize()
    assert torch.equal(view, ref)


def test_reorder_leaves_the_unfilled_part():
    g = torch.Generator().manual_seed(5)
    t0 = torch.randn((2, 4, 3, 50, 8), generator=g)
    par = torch.tensor([[3, 3, 0, 1], [0, 1, 1, 2]], dtype=torch.int32)
    t = t0.to(DEV)
    lmhead.beam_reorder(t[:, :, :, :37], par.to(DEV))
    assert torch.equal(t.cpu()[:, :, :, 37:], t0[:, :, :, 37:])
    assert torch.equal(t.cpu()[:, :, :, :37], plain_reorder(t0[:, :, :, :37], par, 0))


def test_reorder_permuted_and_interleaved_states():
    # keys and values side by side in one tensor, time outside the beams
    g = torch.Generator().manual_seed(6)
    t0 = torch.randn((20, 2, 4, 2, 12), generator=g)          # [time, N, W, k/v, width]
    par = torch.tensor([[1, 0, 3, 3], [2, 2, 2, 0]], dtype=torch.int32)
    t = t0.to(DEV)
    lmhead.beam_reorder([t[:, :, :, 0], t[:, :, :, 1]], par.to(DEV), entry_dim=1)
    assert torch.equal(t.cpu(), plain_reorder(t0, par, 1))


def test_reorder_bad_parents_and_empty():
    t0 = torch.arange(2 * 3 * 4).view(2, 3, 4)
    t = t0.to(DEV)
    par = torch.tensor([[1, -1, 3], [2, 1, 0]], dtype=torch.int32)
    st = torch.zeros(1, dtype=torch.int32, device=DEV)
    lmhead.beam_reorder(t, par.to(DEV), status=st)
    assert int(st.item()) == lmhead.DEV_BAD_PARENT
    ok = torch.tensor([[1, 1, 2], [2, 1, 0]], dtype=torch.int32)
    assert torch.equal(t.cpu(), plain_reorder(t0, ok, 0))
    lmhead.beam_reorder(torch.empty((2, 3, 0), device=DEV), par.to(DEV))


def test_reorder_many_states():
    par = torch.tensor([[1, 0]], dtype=torch.int32, device=DEV)
    states = [torch.tensor([[[float(i)], [-float(i)]]], device=DEV) for i in range(150)]
    lmhead.beam_reorder(states, par)
    assert [s.flatten().tolist() for s in states] == [[-float(i), float(i)] for i in range(150)]


def test_overlapping_state_is_refused():
    par = torch.zeros((2, 3), dtype=torch.int32, device=DEV)
    t = torch.zeros(8, device=DEV)
    with pytest.raises(lmhead.LmhError):
        lmhead.beam_reorder(t.expand(2, 3, 8), par)
    with pytest.raises(ValueError, match="twice"):
        lmhead.beam_reorder([torch.zeros((2, 3, 8), device=DEV)] * 2, par)


# ------------------------------------------------------------------ graphs

def test_captured_and_replayed_step():
    """Selection and reorder in one graph: replays on new logits give what eager calls give."""
    N, W, V, C = 2, 4, 9000, 8
    x, s = data(N, W, V, 21)
    hist = torch.arange(N * W * 6, device=DEV).view(N, W, 6)
    ref_hist = hist.clone()
    out = [torch.empty((N, C), device=DEV), torch.empty((N, C), dtype=torch.int32, device=DEV),
           torch.empty((N, C), dtype=torch.int64, device=DEV), torch.empty((N, W), device=DEV),
           torch.empty((N, W), dtype=torch.int32, device=DEV),
           torch.empty((N, W), dtype=torch.int64, device=DEV)]
    ws = torch.empty(lmhead.beam_select_workspace_bytes(N, W, V, C), dtype=torch.uint8, device=DEV)
    keep = hist.clone()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        lmhead.beam_select(x, s, *out, ws, eos=2)
        lmhead.beam_reorder(hist, out[4])
    hist.copy_(keep)
    for step in range(3):
        x.copy_(data(N, W, V, 30 + step)[0])
        g.replay()
        torch.cuda.synchronize()
        ref = run_select(x, s, C, 2)
        lmhead.beam_reorder(ref_hist, ref[4])
        for a, b in zip(out, ref):
            assert torch.equal(a, b)
        assert torch.equal(hist, ref_hist)
