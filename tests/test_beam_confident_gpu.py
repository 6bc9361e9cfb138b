"""beam_select on rows that one token dominates: the logarithm of the sum, and the order of
beams whose totals lie closer than FP32's step.

Tolerance of a total: the terms of a row's C best logits enter lse in FP64; any other is off by
at most 2^-20 of itself (the base-2 exponential 2^-22, its argument's two roundings, weighted by
the terms they belong to, 2^-22.5, five FP32 additions 5 * 2^-24), so lse by at most 2^-20 of the
share of probability they hold.  The score is rounded to FP32, 2^-24 of itself; FP64's own
roundings stay below 1e-12 at these sizes.
"""
import pytest
import torch

from lm_head_fp32_b200 import lmhead

pytestmark = pytest.mark.gpu
DEV = "cuda"


def select(x, s, C, eos=-1):
    N, W, V = x.shape
    out = [torch.empty((N, C), device=DEV), torch.empty((N, C), dtype=torch.int32, device=DEV),
           torch.empty((N, C), dtype=torch.int64, device=DEV)]
    ws = torch.empty(lmhead.beam_select_workspace_bytes(N, W, V, C), dtype=torch.uint8, device=DEV)
    lmhead.beam_select(x, s, *out, None, None, None, ws, eos=eos)
    torch.cuda.synchronize()
    return out


def confident(N, W, V, seed, dtype):
    """Rows of a low bulk, one likely token, and before it (4096 places: the same thread of a
    part of several batches) one that is 0.7 to 5.4 less likely in the logit."""
    g = torch.Generator(device=DEV).manual_seed(seed)
    x = torch.randn((N, W, V), generator=g, device=DEV) * 2 - 30
    at = torch.randint(0, V - 8192, (N, W, 1), generator=g, device=DEV)
    top = 8 + 4 * torch.rand((N, W, 1), generator=g, device=DEV)
    less = 0.7 + 4.7 * torch.rand((N, W, 1), generator=g, device=DEV)
    x.scatter_(2, at, top - less)
    x.scatter_(2, at + 4096, top)
    return x.to(dtype), (at + 4096)[:, :, 0]


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("N,W,V,C", [(16, 8, 131072, 16), (64, 2, 128257, 4), (2, 2, 40000, 8), (300, 4, 20011, 1)])
def test_scores_of_confident_rows(N, W, V, C, dtype):
    x, top = confident(N, W, V, 5, dtype)
    score, _, token = select(x.view(N * W, 1, V), torch.zeros((N * W, 1), device=DEV), C)
    p = x.double().softmax(2).view(N * W, V)
    best = p.sort(dim=1, descending=True)[0][:, :C]
    assert torch.equal(token[:, 0], top.flatten())
    ref = best[:, 0].log()
    tol = 2.0 ** -20 * (1 - best.sum(1)).clamp(min=0) + 2.0 ** -24 * ref.abs() + 1e-12
    off = (score[:, 0].double() - ref).abs()
    assert (off <= tol).all(), f"worst {float((off / tol).max()):.2f} of the tolerance, {float(off.max()):.1e}"


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("gap", [2e-7, -2e-7])
def test_order_of_close_beams(gap, dtype):
    """Two beams whose best continuations' totals differ by about 2e-7."""
    N, V, C = 64, 131072, 4
    x, top = confident(N, 2, V, 7, dtype)
    logp = x.double().log_softmax(2).gather(2, top[:, :, None])[:, :, 0]
    s = torch.full((N, 2), -0.5, device=DEV)
    s[:, 1] = (s[:, 0].double() + logp[:, 0] - logp[:, 1] + gap).float()
    total = s.double() + logp
    diff = total[:, 1] - total[:, 0]      # s is rounded by at most 2^-24
    assert ((diff - gap).abs() <= 2.0 ** -24).all()
    score, beam, token = select(x, s, C)
    first = (diff > 0).int()
    assert torch.equal(beam[:, 0], first) and torch.equal(beam[:, 1], 1 - first)
    assert torch.equal(token[:, 0], top.gather(1, first.long()[:, None])[:, 0])


@pytest.mark.parametrize("V", [20001, 300001])
def test_sum_over_equal_logits(V):
    # more values at the threshold than a part can list
    N = 64
    logv = torch.tensor(float(V), dtype=torch.float64).log()
    s = logv.float().expand(N, 1).contiguous().to(DEV)
    score = select(torch.full((N, 1, V), -0.5, device=DEV), s, 6)[0]
    ref = float(s[0, 0].double()) - float(logv)
    assert ((score.double() - ref).abs() <= 2.0 ** -24 * abs(ref) + 1e-12).all()
