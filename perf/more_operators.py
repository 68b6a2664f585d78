"""Cases of the operators at a model's ends and between its blocks: what is measured, on which inputs, and the
operators' plain forms.

Operators (``case["op"]``):

* ``loss``: the language-model head and its loss, logits = hidden @ weight.T, softmax cross entropy of each token
  against its target, and the mean.
* ``loss_step``: the same with its gradients, of the hidden states and of the head's weight, times a loss scale that
  lies in device memory (a dynamic loss scaler's).
* ``embed`` / ``embed_grad``: rows of a table by token ids, times a scale, and the table's gradient.
* ``norm`` / ``norm_grad``: layer norm of each row, and the gradients of its input, weight and bias.

Sizes are those of the GPT-2 and Llama-style models of the package's workloads and of other ones between.  Tokens
are Zipf-distributed, as in text.  A target or an id outside the vocabulary marks padding: such a token has no loss,
its embedding is zero, and it takes part in no gradient.  ``shift`` is by how many elements a weight and its
gradient begin after a 256-byte boundary: tensors that follow one another in a flat buffer begin anywhere.
"""
from __future__ import annotations

import math

import torch

own = False

PKG = "zero_partitioned_mixed_replica_gb300"
DT = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
SIZE = {"bf16": 2, "fp16": 2, "fp32": 4}
EPS = 1e-5
PAD = -100
LOSS_SCALE = {"bf16": 1.0, "fp16": 65536.0, "fp32": 1.0}
EMBED_SCALE = 1.25


# -- cases -----------------------------------------------------------------------------------------------
def _case(name, op, n, d, vocab=0, dtype="bf16", padded=0.0, shift=0):
    return {"name": name, "op": op, "n": n, "d": d, "vocab": vocab, "dtype": dtype, "padded": padded, "shift": shift}


def listed():
    return [
        # scoring a short text under a 124M model: latency, the weight is read once
        _case("loss short", "loss", 37, 768, 50257),
        # validation loss of four contexts under the 1.5B model
        _case("loss xl", "loss", 4096, 1600, 50257, "fp16"),
        # fine-tuning a 124M model on one context whose prompt has no loss; an odd number of tokens
        _case("loss step small", "loss_step", 1023, 768, 50257, padded=0.3),
        # a training micro-batch of the 1.5B model: 8 contexts of 1024, fp16 under a loss scale
        _case("loss step xl", "loss_step", 8192, 1600, 50257, "fp16"),
        # and of the 7B model
        _case("loss step 7b", "loss_step", 8192, 4096, 32000),
        # embeddings of 8 contexts
        _case("embed xl", "embed", 8192, 1600, 50257),
        # the embedding's gradient in a fine-tuning step, with padding
        _case("embed grad small", "embed_grad", 1023, 768, 50257, padded=0.2),
        # and in a step of 32 contexts of the 1.5B model
        _case("embed grad xl", "embed_grad", 32768, 1600, 50257),
        # a norm for a few tokens: latency
        _case("norm small", "norm", 64, 768),
        # every norm of a training forward pass, 32 contexts
        _case("norm xl", "norm", 32768, 1600),
        # a model with odd widths kept in fp32, its parameters gapless in one buffer
        _case("norm grad odd", "norm_grad", 1021, 1001, dtype="fp32", shift=3),
        # every norm of a training backward pass, 32 contexts
        _case("norm grad xl", "norm_grad", 32768, 1600),
    ]


def draw(rng):
    log = lambda a, b: int(round(math.exp(rng.uniform(math.log(a), math.log(b)))))  # noqa: E731
    op = rng.choice(["loss", "loss_step", "loss_step", "embed", "embed_grad", "embed_grad", "norm", "norm_grad", "norm_grad"])
    while True:
        d = log(8, 4096)
        if rng.random() < 0.7:           # widths are mostly multiples of something
            d = max(8, d // 64 * 64 if d >= 256 else d // 8 * 8)
        vocab = log(16, 50257)
        n = log(1, 8192 if op.startswith("loss") else 32768)
        if op.startswith("norm"):
            vocab = 0
            if n * d <= 32768 * 1600:
                break
        elif n * vocab * d <= 8192 * 32000 * 4096 and max(n, vocab) * d <= 50257 * 1600 * 2:
            break
    dtype = rng.choice(["bf16", "bf16", "fp16"] if op.startswith("loss") else ["bf16", "bf16", "fp16", "fp32"])
    c = _case(None, op, n, d, vocab, dtype, rng.choice([0.0, 0.0, 0.25, 0.9]) if vocab and n > 4 else 0.0,
              rng.choice([0, 0, 0, 1, 5, 8]))
    del c["name"]
    return c


def work(case):
    n, d, v, op = case["n"], case["d"], case["vocab"], case["op"]
    s = SIZE[case["dtype"]]
    if op == "loss":
        return {"bytes": (n + v) * d * s + 12 * n, "flops": 2 * n * v * d}
    if op == "loss_step":     # three products; a second one for the logits is the price of not keeping them
        return {"bytes": 2 * (n + v) * d * s + 12 * n, "flops": 6 * n * v * d}
    if op == "embed":
        return {"bytes": n * (2 * d * s + 8), "flops": n * d}
    if op == "embed_grad":
        return {"bytes": n * (d * s + 8) + v * d * s, "flops": n * d}
    if op == "norm":
        return {"bytes": 2 * n * d * s + 2 * d * s + 8 * n, "flops": 8 * n * d}
    return {"bytes": 3 * n * d * s + 3 * d * s + 8 * n, "flops": 14 * n * d}


# -- inputs ----------------------------------------------------------------------------------------------
def _inputs(case, seed, dev="cuda"):
    n, d, v, op, dt = case["n"], case["d"], case["vocab"], case["op"], DT[case["dtype"]]
    gen = torch.Generator(dev).manual_seed(seed)
    randn = lambda *s: torch.randn(*s, generator=gen, device=dev)  # noqa: E731
    rand = lambda *s: torch.rand(*s, generator=gen, device=dev)  # noqa: E731

    def placed(t):      # as a tensor of a flat buffer
        flat = torch.zeros(t.numel() + case["shift"], dtype=dt, device=dev)
        flat[case["shift"]:].copy_(t.reshape(-1))
        return flat[case["shift"]:].view(t.shape)

    s = {}
    if v:
        # token k (from 0) about as often as 1 / (k + 1)
        ids = (torch.exp(rand(n).double() * math.log(v + 1)).long() - 1).clamp_(0, v - 1)
        pad = rand(n) < case["padded"]
    if op in ("loss", "loss_step"):
        w = placed(randn(v, d) * 0.02)
        s["weight"] = w
        # a half-trained model: the hidden state leans towards its target's row
        lean = w[ids].float()
        lean /= lean.norm(dim=1, keepdim=True).clamp_(min=1e-6)
        s["hidden"] = (randn(n, d) + 6.0 * rand(n, 1) * math.sqrt(1600 / d) * lean).to(dt)
        s["targets"] = torch.where(pad, PAD, ids)
        s["scale"] = torch.full((1,), LOSS_SCALE[case["dtype"]], device=dev)
    elif op in ("embed", "embed_grad"):
        s["ids"] = torch.where(pad, PAD, ids)
        if op == "embed":
            s["weight"] = placed(randn(v, d) * 0.02)
        else:
            s["grad"] = (randn(n, d) * 1e-2).to(dt)
            s["grad_weight"] = placed(torch.zeros(v, d, device=dev))
    else:
        s["weight"], s["bias"] = placed(1.0 + 0.1 * randn(d)), placed(0.1 * randn(d))
        # a residual stream: some channels are large everywhere
        s["x"] = (randn(n, d) * 1.5 + 2.0 * randn(d)).to(dt)
        if op == "norm_grad":
            s["grad"] = (randn(n, d) * 1e-2).to(dt)
            x = s["x"].double() if case["dtype"] == "fp32" else s["x"].float()
            mean = x.mean(1)
            s["mean"] = mean.float()
            s["rstd"] = ((x - mean[:, None]).square().mean(1) + EPS).rsqrt().float()
            del x
            s["grad_weight"], s["grad_bias"] = placed(torch.zeros(d, device=dev)), placed(torch.zeros(d, device=dev))
    if op == "loss_step":
        s["grad_weight"] = placed(torch.zeros(v, d, device=dev))
    return s


def prepare(case, seed):
    s = _inputs(case, seed)
    s["case"] = case
    return s


# -- the operators ---------------------------------------------------------------------------------------
def run(state):
    return _run_own(state) if own else _run_plain(state)


def _run_own(s):
    from zero_partitioned_mixed_replica_gb300 import layers
    op = s["case"]["op"]
    if op in ("loss", "loss_step"):
        loss, losses, saved = layers.lm_loss_forward(s["hidden"], s["weight"], s["targets"])
        if op == "loss":
            return {"loss": loss, "losses": losses}
        grad_hidden = layers.lm_loss_backward(s["hidden"], s["weight"], s["targets"], saved, s["grad_weight"], scale=s["scale"])
        return {"loss": loss, "losses": losses, "grad_hidden": grad_hidden, "grad_weight": s["grad_weight"]}
    if op == "embed":
        return {"out": layers.embedding_forward(s["weight"], s["ids"], scale=EMBED_SCALE)}
    if op == "embed_grad":
        layers.embedding_backward(s["grad"], s["ids"], s["grad_weight"], scale=EMBED_SCALE)
        return {"grad_weight": s["grad_weight"]}
    if op == "norm":
        y, mean, rstd = layers.layer_norm_forward(s["x"], s["weight"], s["bias"], eps=EPS)
        return {"y": y, "mean": mean, "rstd": rstd}
    grad_x = layers.layer_norm_backward(s["grad"], s["x"], s["weight"], s["mean"], s["rstd"], s["grad_weight"], s["grad_bias"])
    return {"grad_x": grad_x, "grad_weight": s["grad_weight"], "grad_bias": s["grad_bias"]}


def _run_plain(s):
    case = s["case"]
    op, dt = case["op"], DT[case["dtype"]]
    if op in ("loss", "loss_step"):
        hidden, weight, targets = s["hidden"].float(), s["weight"].float(), s["targets"]
        counted = (targets >= 0) & (targets < case["vocab"])
        at = torch.where(counted, targets, 0)[:, None]
        share = 1.0 / counted.sum().clamp(min=1).float()
        logits = hidden @ weight.t()
        chosen = logits.gather(1, at)[:, 0]
        top = logits.amax(1, keepdim=True)
        logits = torch.exp(logits - top)
        total = logits.sum(1, keepdim=True)
        losses = torch.where(counted, torch.log(total[:, 0]) + top[:, 0] - chosen, 0.0)
        out = {"loss": (losses.double().sum() * share).float(), "losses": losses}
        if op == "loss":
            return out
        logits /= total
        logits.scatter_add_(1, at, torch.full_like(total, -1.0))
        logits *= (counted * share)[:, None]
        out["grad_hidden"] = ((logits @ weight) * s["scale"]).to(dt)
        out["grad_weight"] = ((logits.t() @ hidden) * s["scale"]).to(dt)
        return out
    if op in ("embed", "embed_grad"):
        ids = s["ids"]
        inside = (ids >= 0) & (ids < case["vocab"])
        at = torch.where(inside, ids, 0)
        if op == "embed":
            return {"out": torch.where(inside[:, None], s["weight"][at].float() * EMBED_SCALE, 0.0).to(dt)}
        rows = torch.where(inside[:, None], s["grad"].float() * EMBED_SCALE, 0.0)
        # in 64 bits where a token is often: sums of many terms in an order that changes
        wide = torch.float64 if case["dtype"] == "fp32" else torch.float32
        grad = torch.zeros(case["vocab"], case["d"], dtype=wide, device=ids.device)
        return {"grad_weight": grad.index_add_(0, at, rows.to(wide)).to(dt)}
    x = s["x"].float()
    if op == "norm":
        mean = x.mean(1, keepdim=True)
        x = x - mean
        rstd = 1.0 / torch.sqrt(x.square().mean(1, keepdim=True) + EPS)
        y = x * rstd * s["weight"].float() + s["bias"].float()
        return {"y": y.to(dt), "mean": mean[:, 0], "rstd": rstd[:, 0]}
    rstd = s["rstd"][:, None]
    x = (x - s["mean"][:, None]) * rstd
    g = s["grad"].float()
    gw = g * s["weight"].float()
    grad_x = (gw - gw.mean(1, keepdim=True) - x * (gw * x).mean(1, keepdim=True)) * rstd
    return {"grad_x": grad_x.to(dt), "grad_weight": (g * x).sum(0).to(dt), "grad_bias": g.sum(0).to(dt)}


# -- the definition in 64 bits ---------------------------------------------------------------------------
def exact(case, seed):
    d = _inputs(case, seed)
    op, v = case["op"], case["vocab"]
    if op in ("loss", "loss_step"):
        hidden, weight = d["hidden"].double(), d["weight"].double()
        keep = [0 <= t < v for t in d["targets"].tolist()]
        count = max(1, sum(keep))
        keep = torch.tensor(keep, dtype=torch.float64, device=hidden.device)
        losses = torch.zeros(case["n"], dtype=torch.float64, device=hidden.device)
        gh, gw = torch.zeros_like(hidden), torch.zeros_like(weight)
        for a in range(0, case["n"], 1024):
            z = hidden[a:a + 1024] @ weight.T
            target = torch.zeros_like(z)
            row = torch.nonzero(keep[a:a + 1024])[:, 0]
            target[row, d["targets"][a:a + 1024][row]] = 1.0
            lse = torch.logsumexp(z, 1)
            losses[a:a + 1024] = (lse - (z * target).sum(1)) * keep[a:a + 1024]
            if op == "loss_step":
                dz = (torch.softmax(z, 1) - target) * (keep[a:a + 1024] * LOSS_SCALE[case["dtype"]] / count)[:, None]
                gh[a:a + 1024] = dz @ weight
                gw += dz.T @ hidden[a:a + 1024]
        out = {"loss": losses.sum() / count, "losses": losses}
        return out if op == "loss" else {**out, "grad_hidden": gh, "grad_weight": gw}
    if op == "embed":
        table = torch.cat([d["weight"].double() * EMBED_SCALE, torch.zeros(1, case["d"], dtype=torch.float64, device="cuda")])
        return {"out": table[torch.where(d["ids"] < 0, v, d["ids"])]}
    if op == "embed_grad":
        # the sorted tokens' running sums at the ends of each id's stretch
        order = torch.argsort(d["ids"], stable=True)
        ids = d["ids"][order]
        total = torch.cumsum(d["grad"][order].double() * EMBED_SCALE, 0)
        total = torch.cat([torch.zeros(1, case["d"], dtype=torch.float64, device="cuda"), total])
        edges = torch.searchsorted(ids, torch.arange(v + 1, device="cuda"))
        return {"grad_weight": total[edges[1:]] - total[edges[:-1]]}
    x, w = d["x"].double(), d["weight"].double()
    if op == "norm":
        var, mean = torch.var_mean(x, 1, unbiased=False)
        rstd = (var + EPS) ** -0.5
        return {"y": (x - mean[:, None]) * rstd[:, None] * w + d["bias"].double(), "mean": mean, "rstd": rstd}
    g, rstd = d["grad"].double(), d["rstd"].double()[:, None]
    unit = (x - d["mean"].double()[:, None]) * rstd
    along = torch.einsum("nd,nd,d->n", g, unit, w)[:, None] / case["d"]
    grad_x = rstd * (g * w - (g @ w)[:, None] / case["d"] - unit * along)
    return {"grad_x": grad_x, "grad_weight": torch.einsum("nd,nd->d", g, unit), "grad_bias": g.sum(0)}
