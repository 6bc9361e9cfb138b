"""Timed cases of the decode and fine-tuning operators around the LM head.

Operators (see ``lm_head_fp32_b200.lmhead``):

  adapter_fwd   logits = X . W^T + s_a (X . A_a^T) . B_a^T, the adapter a chosen per token
  adapter_bwd   its gradients: dX, and dA, dB of every adapter
  beam_select   the best continuations over beams and vocabulary, and the beams that go on
  beam_reorder  the beams' states put in the order of their parents, in place

``run`` computes them in elementary torch operations where ``own`` is false, and through this
package's calls where it is true.
"""
import math

import torch

own = False

DEV = "cuda"


# ------------------------------------------------------------------ cases

def listed():
    return [
        # one token of a chat request that has an adapter: the latency of a decode step
        dict(name="adapter_fwd one token", op="adapter_fwd", M=1, K=4096, V=32768, N=4, R=8,
             order="random", out="f32"),
        # a decode batch: 64 requests, each with its own of 32 adapters or none
        dict(name="adapter_fwd decode 64", op="adapter_fwd", M=64, K=4096, V=128256, N=32, R=16,
             order="random", out="f32"),
        # prompts of several requests one behind the other, an odd vocabulary, BF16 logits
        dict(name="adapter_fwd ragged prompts", op="adapter_fwd", M=1021, K=2048, V=32771, N=8, R=64,
             order="runs", out="bf16"),
        # a training or scoring batch with a few adapters: the largest projection
        dict(name="adapter_fwd 4096 tokens", op="adapter_fwd", M=4096, K=4096, V=128256, N=8, R=16,
             order="runs", out="f32"),
        # fine-tuning several adapters at once, mid-size vocabulary
        dict(name="adapter_bwd mid-size", op="adapter_bwd", M=1024, K=4096, V=32768, N=4, R=16,
             order="runs", out="f32"),
        # the same with the large vocabulary, wider adapters and tokens in no order
        dict(name="adapter_bwd 4096 tokens", op="adapter_bwd", M=4096, K=4096, V=128256, N=8, R=32,
             order="random", out="bf16"),
        # one request with four beams: the latency of a search step
        dict(name="beam_select one request", op="beam_select", N=1, W=4, V=32768, dtype="f32"),
        # a service's batch
        dict(name="beam_select 16 x 4", op="beam_select", N=16, W=4, V=128256, dtype="f32"),
        # odd sizes and BF16 logits
        dict(name="beam_select odd bf16", op="beam_select", N=7, W=5, V=32771, dtype="bf16"),
        # offline search with wide beams over a large vocabulary
        dict(name="beam_select 64 x 8", op="beam_select", N=64, W=8, V=151936, dtype="f32"),
        # the token history of a few requests: 8-byte elements, odd row length
        dict(name="beam_reorder history", op="beam_reorder", N=5, W=4, outer=1, heads=1, used=333,
             room=512, width=1, dtype="i64", states=1),
        # key and value caches of eight layers, filled to 1000 of 1024 places
        dict(name="beam_reorder caches", op="beam_reorder", N=16, W=4, outer=1, heads=8, used=1000,
             room=1024, width=128, dtype="bf16", states=16),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["adapter_fwd", "adapter_bwd", "beam_select", "beam_reorder"])
    if op in ("adapter_fwd", "adapter_bwd"):
        M = _log_int(rng, 1, 4096) if op == "adapter_fwd" else _log_int(rng, 16, 4096)
        K = 8 * _log_int(rng, 64, 512)
        V = _log_int(rng, 4096, 128256)
        if op == "adapter_bwd":
            V = V // 8 * 8
        return dict(op=op, M=M, K=K, V=V, N=_log_int(rng, 1, 32), R=rng.choice([8, 16, 24, 32, 64]),
                    order=rng.choice(["random", "runs"]), out=rng.choice(["f32", "bf16"]))
    if op == "beam_select":
        return dict(op=op, N=_log_int(rng, 1, 64), W=rng.randint(1, 8), V=_log_int(rng, 1000, 151936),
                    dtype=rng.choice(["f32", "bf16"]))
    used = _log_int(rng, 1, 1000)
    dtype = rng.choice(["bf16", "f32", "i64"])
    return dict(op=op, N=_log_int(rng, 1, 16), W=rng.randint(2, 8), outer=rng.choice([1, 2]),
                heads=rng.randint(1, 8), used=used, room=used + rng.choice([0, 1, 24]),
                width={"bf16": rng.choice([64, 128]), "f32": rng.choice([1, 33]), "i64": 1}[dtype],
                dtype=dtype, states=_log_int(rng, 1, 16))


# ------------------------------------------------------------------ inputs

def _gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed * 1000003 + 17)
    return g


def _normal(g, shape, std, dtype=torch.bfloat16):
    """N(0, std^2) in `dtype`, drawn in slices so that large tensors need no second copy."""
    out = torch.empty(shape, dtype=dtype, device=DEV)
    flat = out.view(-1)
    for i in range(0, flat.numel(), 1 << 28):
        part = flat[i:i + (1 << 28)]
        part.copy_(torch.randn(part.numel(), generator=g, device=DEV).mul_(std))
    return out


def _adapter_ids(g, M, N, order):
    """One adapter id per token, -1 for none (about one token in eight)."""
    a = torch.randint(0, N, (M,), generator=g, device=DEV, dtype=torch.int32)
    none = torch.rand(M, generator=g, device=DEV) < 0.125
    if order == "runs":
        a, _ = a.sort()
        none = torch.zeros_like(none)
        none[M - M // 8:] = True  # the last request has no adapter
    a[none] = -1
    return a


def _beam_logits(g, rows, V, dtype):
    """Logits of a trained head: a normal bulk and a few likely tokens in each row."""
    x = torch.randn((rows, V), generator=g, device=DEV).mul_(2.5)
    at = torch.randint(0, V // 12, (rows, 12), generator=g, device=DEV)
    at += V // 12 * torch.arange(12, device=DEV)  # twelve different tokens
    x.scatter_add_(1, at, torch.rand((rows, 12), generator=g, device=DEV) * 9)
    return x.to(dtype)


def prepare(case, seed):
    c, g = case, _gen(seed)
    dt = {"f32": torch.float32, "bf16": torch.bfloat16, "i64": torch.int64}
    s = dict(case=c, status=torch.zeros(1, dtype=torch.int32, device=DEV))
    if c["op"] in ("adapter_fwd", "adapter_bwd"):
        M, K, V, N, R = (c[k] for k in "MKVNR")
        s["X"] = _normal(g, (M, K), 1.0)
        s["W"] = _normal(g, (V, K), 0.02)
        s["A"] = _normal(g, (N, R, K), K ** -0.5)
        s["B"] = _normal(g, (N, V, R), 0.02)
        s["scale"] = torch.rand(N, generator=g, device=DEV) + 0.5
        s["adapter"] = _adapter_ids(g, M, N, c["order"])
        if c["op"] == "adapter_fwd":
            s["u"] = torch.empty((M, R), device=DEV)
            s["logits"] = torch.empty((M, V), dtype=dt[c["out"]], device=DEV)
        else:
            # the gradient that a cross-entropy over M tokens hands back
            dl = torch.empty((M, V), dtype=torch.bfloat16, device=DEV)
            y = torch.randint(0, V, (M,), generator=g, device=DEV)
            for i in range(0, M, 512):
                p = torch.randn((min(512, M - i), V), generator=g, device=DEV).mul_(1.3).softmax(1)
                p.scatter_add_(1, y[i:i + 512, None], torch.full_like(p[:, :1], -1.0))
                dl[i:i + 512] = p.div_(M)
            s["dlogits"] = dl
            # saved by the forward pass
            s["u"] = _masked(s, (s["X"].float() @ s["A"].float().view(N * R, K).T)) \
                .view(M, N, R).sum(1)
            s["g"] = torch.empty((M, R), device=DEV)
            s["dX"] = torch.empty((M, K), dtype=dt[c["out"]], device=DEV)
            s["dA"] = torch.empty((N, R, K), device=DEV)
            s["dB"] = torch.empty((N, V, R), device=DEV)
    elif c["op"] == "beam_select":
        N, W, V = c["N"], c["W"], c["V"]
        s["logits"] = _beam_logits(g, N * W, V, dt[c["dtype"]]).view(N, W, V)
        s["scores"] = -15 - 3 * torch.rand((N, W), generator=g, device=DEV)
        s["eos"] = 2
        C = 2 * W
        f = dict(device=DEV)
        s["out"] = (torch.empty((N, C), **f), torch.empty((N, C), dtype=torch.int32, **f),
                    torch.empty((N, C), dtype=torch.int64, **f), torch.empty((N, W), **f),
                    torch.empty((N, W), dtype=torch.int32, **f),
                    torch.empty((N, W), dtype=torch.int64, **f))
    else:
        N, W = c["N"], c["W"]
        shape = (c["outer"], N, W, c["heads"], c["room"], c["width"])
        made = []
        for _ in range(c["states"]):
            if c["dtype"] == "i64":
                made.append(torch.randint(0, 1 << 40, shape, generator=g, device=DEV))
            else:
                made.append(_normal(g, shape, 1.0, dt[c["dtype"]]))
        # the filled places of each cache
        s["states"] = [t[:, :, :, :, :c["used"]] for t in made]
        s["parents"] = torch.randint(0, W, (N, W), generator=g, device=DEV, dtype=torch.int32)
    return s


# ------------------------------------------------------------------ the plain forms

def _masked(s, t):
    """t [M, N * R], with scale where the columns are of the token's adapter and 0 elsewhere."""
    N = s["scale"].numel()
    hot = (s["adapter"][:, None] == torch.arange(N, device=DEV)[None]) * s["scale"]
    return (t.view(t.shape[0], N, -1) * hot[:, :, None]).view(t.shape)


def _plain_adapter_fwd(s):
    N, R, K = s["A"].shape
    X = s["X"].float()
    u = _masked(s, X @ s["A"].float().view(N * R, K).T)
    logits = X @ s["W"].float().T
    logits += u @ s["B"].float().transpose(1, 2).reshape(N * R, -1)
    return {"logits": logits.to(s["logits"].dtype), "u": u.view(-1, N, R).sum(1)}


def _plain_adapter_bwd(s):
    N, R, K = s["A"].shape
    M, V = s["dlogits"].shape
    dl, X = s["dlogits"].float(), s["X"].float()
    A = s["A"].float().view(N * R, K)
    g = _masked(s, dl @ s["B"].float().transpose(1, 2).reshape(N * R, V).T)
    dX = dl @ s["W"].float() + g @ A
    hot = (s["adapter"][:, None] == torch.arange(N, device=DEV)[None]).float()
    u = (s["u"][:, None] * hot[:, :, None]).view(M, N * R)
    dA = (g.T @ X).view(N, R, K)
    dB = (dl.T @ u).view(V, N, R).transpose(0, 1).contiguous()
    return {"dX": dX.to(s["dX"].dtype), "g": g.view(M, N, R).sum(1), "dA": dA, "dB": dB}


def _plain_beam_select(s):
    # in 64 bits: which of two continuations is ahead goes by their last places
    N, W, V = s["logits"].shape
    C = 2 * W
    x = s["logits"].double()
    m = x.amax(2, keepdim=True)
    x = x - m
    total = s["scores"].double()[:, :, None] + x - x.exp().sum(2, keepdim=True).log()
    score, flat = total.view(N, W * V).sort(dim=1, descending=True, stable=True)
    score, flat = score[:, :C], flat[:, :C]
    beam, token = flat // V, flat % V
    # the first W candidates that do not end their sequence go on
    keep = (token == s["eos"]).int().sort(dim=1, stable=True)[1][:, :W]
    return [score.float(), beam.int(), token, score.gather(1, keep).float(),
            beam.gather(1, keep).int(), token.gather(1, keep)]


def _plain_beam_reorder(s):
    N, W = s["parents"].shape
    at = s["parents"].long() + W * torch.arange(N, device=DEV)[:, None]
    for t in s["states"]:
        t.copy_(t.flatten(1, 2)[:, at.view(-1)].view(t.shape))
    return s["states"]


# ------------------------------------------------------------------ one pass

def run(state):
    s = state
    op = s["case"]["op"]
    if not own:
        return {"adapter_fwd": _plain_adapter_fwd, "adapter_bwd": _plain_adapter_bwd,
                "beam_select": _plain_beam_select, "beam_reorder": _plain_beam_reorder}[op](s)
    from lm_head_fp32_b200 import lmhead
    if op in ("adapter_fwd", "adapter_bwd"):
        N, R, K = s["A"].shape
        if "workspace" not in s:
            n = lmhead.lmhead_lora_workspace_bytes(s["X"].shape[0], K, s["W"].shape[0], R, N)
            s["workspace"] = torch.empty(n, dtype=torch.uint8, device=DEV)
        if op == "adapter_fwd":
            lmhead.lmhead_fwd_lora(s["X"], s["W"], s["A"], s["B"], s["scale"], s["adapter"], s["u"],
                                   s["logits"], s["workspace"], s["status"])
            return {"logits": s["logits"], "u": s["u"]}
        lmhead.lmhead_bwd_dx_lora(s["dlogits"], s["W"], s["A"], s["B"], s["scale"], s["adapter"],
                                  s["g"], s["dX"], s["workspace"], s["status"])
        lmhead.lmhead_bwd_lora(s["dlogits"], s["X"], s["u"], s["g"], s["adapter"], s["dA"], s["dB"],
                               s["workspace"], s["status"])
        return {"dX": s["dX"], "g": s["g"], "dA": s["dA"], "dB": s["dB"]}
    if op == "beam_select":
        if "workspace" not in s:
            N, W, V = s["logits"].shape
            n = lmhead.beam_select_workspace_bytes(N, W, V, 2 * W)
            s["workspace"] = torch.empty(n, dtype=torch.uint8, device=DEV)
        lmhead.beam_select(s["logits"], s["scores"], *s["out"], s["workspace"], eos=s["eos"],
                           status=s["status"])
        return list(s["out"])
    lmhead.beam_reorder(s["states"], s["parents"], entry_dim=1, status=s["status"])
    return s["states"]


def work(case):
    c = case
    if c["op"] in ("adapter_fwd", "adapter_bwd"):
        M, K, V, N, R = (c[k] for k in "MKVNR")
        out = 4 if c["out"] == "f32" else 2
        ad = min(M, N)  # adapters that some token uses
        shared = 2 * (M * K + V * K) + 2 * ad * R * (K + V) + 4 * M + 4 * N
        if c["op"] == "adapter_fwd":
            return {"bytes": shared + M * V * out + 4 * M * R,
                    "flops": 2.0 * M * V * K + 2.0 * M * R * (K + V)}
        return {"bytes": shared + 2 * M * V + out * M * K + 4 * N * R * (K + V) + 8 * M * R,
                "flops": 2.0 * M * V * K + 4.0 * M * R * (K + V)}
    if c["op"] == "beam_select":
        N, W, V = c["N"], c["W"], c["V"]
        return {"bytes": N * W * V * (4 if c["dtype"] == "f32" else 2) + N * W * (4 + 3 * 16),
                "flops": 3.0 * N * W * V}
    # with parents drawn evenly: W - 1 of W rows change, and a row is read if another one wants it
    W = c["W"]
    row = c["outer"] * c["heads"] * c["used"] * c["width"] * {"bf16": 2, "f32": 4, "i64": 8}[c["dtype"]]
    moved = (W - 1) + W * (1 - (1 - 1 / W) ** (W - 1))
    return {"bytes": c["states"] * c["N"] * row * moved + 4 * c["N"] * W, "flops": 0}


# ------------------------------------------------------------------ from the definitions, in 64 bits

def exact(case, seed):
    c = case
    if c["op"] == "beam_reorder":
        return None  # values are moved, none is computed
    s = prepare(case, seed)
    if c["op"] == "beam_select":
        N, W, V = c["N"], c["W"], c["V"]
        rows = []
        for n in range(N):
            logp = torch.log_softmax(s["logits"][n].double(), dim=1) + s["scores"][n].double()[:, None]
            best = logp.reshape(-1).topk(2 * W)
            rest = best.values[best.indices % V != s["eos"]][:W]
            rows.append((best.values, rest))
        return [torch.stack([r[0] for r in rows]), None, None, torch.stack([r[1] for r in rows]),
                None, None]
    # adapter by adapter
    X = s["X"].double()
    if c["op"] == "adapter_fwd":
        out = X @ s["W"].double().T
        u = torch.zeros((c["M"], c["R"]), dtype=torch.float64, device=DEV)
    else:
        dl = s["dlogits"].double()
        out = dl @ s["W"].double()
        u = torch.zeros((c["M"], c["R"]), dtype=torch.float64, device=DEV)
        dA = torch.zeros(s["A"].shape, dtype=torch.float64, device=DEV)
        dB = torch.zeros(s["B"].shape, dtype=torch.float64, device=DEV)
    for a in range(c["N"]):
        at = torch.nonzero(s["adapter"] == a).view(-1)
        if not at.numel():
            continue
        A, B, sc = s["A"][a].double(), s["B"][a].double(), s["scale"][a].double()
        if c["op"] == "adapter_fwd":
            u[at] = sc * (X[at] @ A.T)
            out[at] += u[at] @ B.T
        else:
            d = dl[at]
            u[at] = sc * (d @ B)
            out[at] += u[at] @ A
            dA[a] = u[at].T @ X[at]
            dB[a] = d.T @ s["u"][at].double()
    if c["op"] == "adapter_fwd":
        return {"logits": out, "u": u}
    return {"dX": out, "g": u, "dA": dA, "dB": dB}
