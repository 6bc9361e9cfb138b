"""The loss entries give every gradient that is asked for, or refuse: none is dropped."""
import pytest
import torch

from lm_head_fp32_b200 import loss, synth

B16 = torch.bfloat16


def inputs(device="cuda", M=150, K=128, V=1000, R=16, N=3):
    g = torch.Generator().manual_seed(3)

    def nrm(*shape, std=1.0):
        return (torch.randn(shape, generator=g) * std).to(B16).to(device)

    X, W = nrm(M, K), nrm(V, K, std=0.1)
    A, B = nrm(N, R, K, std=K ** -0.5), nrm(N, V, R, std=0.1)
    scale = (torch.rand(N, generator=g) + 0.5).to(device)
    ids = torch.randint(-1, N, (M,), generator=g, dtype=torch.int32).to(device)
    return X, W, A, B, scale, ids, synth.targets(M, V, 0.1, 9).to(device)


def test_a_scale_that_asks_for_a_gradient_is_refused():
    X, W, A, B, scale, ids, t = inputs("cpu")
    with pytest.raises(ValueError, match="scale"):
        loss.lm_head_lora_cross_entropy(X, W, A, B, scale.requires_grad_(), ids, t)
    # nobody asks for it here: on to the next check, that of the device
    with torch.no_grad(), pytest.raises(ValueError, match="CUDA"):
        loss.lm_head_lora_cross_entropy(X, W, A, B, scale, ids, t)
    with pytest.raises(ValueError, match="CUDA"):
        loss.lm_head_lora_cross_entropy(X, W, A, B, scale.detach(), ids, t)


@pytest.mark.gpu
def test_a_scale_that_asks_is_taken_without_gradients():
    X, W, A, B, scale, ids, t = inputs()
    ref = loss.lm_head_lora_cross_entropy(X, W, A, B, scale, ids, t)
    with torch.no_grad():
        assert torch.equal(loss.lm_head_lora_cross_entropy(X, W, A, B, scale.requires_grad_(), ids, t), ref)


@pytest.mark.gpu
@pytest.mark.parametrize("wants", ["A", "B", "AB", "X", "W", "XWAB"])
def test_gradients_asked_for_alone_are_those_of_all(wants):
    """Frozen features, a frozen head or frozen adapters: what is asked for comes, the same
    bits as with everything asked for, and nothing else."""
    X, W, A, B, scale, ids, t = inputs()

    def grads(names):
        p = {k: v.clone().requires_grad_(k in names) for k, v in zip("XWAB", (X, W, A, B))}
        loss.lm_head_lora_cross_entropy(*p.values(), scale, ids, t).sum().backward()
        return {k: v.grad for k, v in p.items()}

    every, got = grads("XWAB"), grads(wants)
    for k in "XWAB":
        assert (got[k] is None) == (k not in wants)
        assert got[k] is None or torch.equal(got[k], every[k])


@pytest.mark.gpu
@pytest.mark.parametrize("lora", [False, True])
def test_a_second_derivative_is_refused(lora):
    X, W, A, B, scale, ids, t = inputs()
    leaves = [p.requires_grad_() for p in ((X, W, A, B) if lora else (X, W))]

    def out():
        return (loss.lm_head_lora_cross_entropy(X, W, A, B, scale, ids, t) if lora
                else loss.lm_head_cross_entropy(X, W, t)).sum()

    ref = torch.autograd.grad(out(), leaves)
    got = torch.autograd.grad(out(), leaves, create_graph=True)
    for r, g in zip(ref, got):
        assert torch.equal(r, g)          # the first derivative as ever
        with pytest.raises(RuntimeError, match="once"):
            (X.float().sum() + g.float().pow(2).sum()).backward(retain_graph=True)
