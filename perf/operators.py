"""The operators at the answer end of the stack, as cases to measure: layer norm, log probabilities of
given tokens (with entropy and top alternatives) and distillation from a teacher's top logits, each
forward and backward.

`run` computes a case in plain torch (32 bits, rounded once at the end) or, where `own` is set, through
this repository's package. `exact` computes it in 64 bits from the definitions.
"""

import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
SIZE = {"bf16": 2, "fp16": 2, "fp32": 4}
EPS = 1e-6

NORM_ELEMENTS = 8192 * 7168      # the largest layer norm
LOGIT_BYTES = 8192 * 131072 * 2  # the largest logits


def listed():
    return [
        # One decoded token through the norm after the pre-map: latency.
        dict(name="norm_decode", op="norm", T=1, H=7168, dtype="bf16", weights="bf16", bias=True, gap=0),
        # The same norm over a training batch.
        dict(name="norm_batch", op="norm", T=8192, H=7168, dtype="bf16", weights="fp32", bias=True, gap=0),
        # Its gradient over that batch, weights' gradients included.
        dict(name="norm_grad_batch", op="norm_grad", T=8192, H=7168, dtype="bf16", weights="fp32",
             bias=True, gap=0),
        # Odd width and ragged batch, 32-bit activations.
        dict(name="norm_grad_odd", op="norm_grad", T=3001, H=1001, dtype="fp32", weights="fp32",
             bias=True, gap=0),
        # Serving: four sequences' next-token distributions with 20 alternatives.
        dict(name="logprob_decode", op="logprob", T=4, V=131072, dtype="bf16", K=20, entropy=True,
             temperature=0.7, masked=False, pad=0),
        # Serving: a prompt's log probabilities under a grammar's mask, odd vocabulary, 5 alternatives.
        dict(name="logprob_prompt", op="logprob", T=1500, V=100003, dtype="bf16", K=5, entropy=False,
             temperature=1.0, masked=True, pad=0),
        # Training: log probability and entropy of a whole batch's tokens.
        dict(name="logprob_batch", op="logprob", T=8192, V=131072, dtype="bf16", K=0, entropy=True,
             temperature=1.0, masked=False, pad=0),
        # The gradient of that batch.
        dict(name="logprob_grad_batch", op="logprob_grad", T=8192, V=131072, dtype="bf16", K=0,
             entropy=True, temperature=1.0, masked=False, pad=0),
        # A ragged batch in 32 bits, vocabulary rows padded to a multiple of 128.
        dict(name="logprob_grad_padded", op="logprob_grad", T=777, V=50021, dtype="fp32", K=0,
             entropy=False, temperature=1.0, masked=False, pad=27),
        # Distillation of a batch from a teacher's 64 best.
        dict(name="distill_batch", op="distill", T=4096, V=131072, dtype="bf16", K=64, temperature=2.0,
             masked=False, pad=0, ragged=False),
        dict(name="distill_grad_batch", op="distill_grad", T=4096, V=131072, dtype="bf16", K=64,
             temperature=2.0, masked=False, pad=0, ragged=False),
        # A small ragged batch whose teacher kept fewer than K tokens in some rows.
        dict(name="distill_grad_ragged", op="distill_grad", T=333, V=32003, dtype="fp16", K=17,
             temperature=1.0, masked=False, pad=0, ragged=True),
    ]


def _spread(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["norm", "norm_grad", "logprob", "logprob_grad", "distill", "distill_grad"])
    dtype = rng.choice(["bf16", "bf16", "fp16", "fp32"])
    if op.startswith("norm"):
        H = _spread(rng, 64, 16384)
        if rng.random() < 0.6:
            H = max(64, H // 64 * 64)
        T = _spread(rng, 1, max(1, min(16384, NORM_ELEMENTS // H * 2 // SIZE[dtype])))
        return dict(op=op, T=T, H=H, dtype=dtype, weights=rng.choice(["fp32", dtype]),
                    bias=rng.random() < 0.7, gap=rng.choice([0, 0, 1, 3]) * H)
    V = _spread(rng, 1000, 160000)
    if rng.random() < 0.5:
        V = max(1024, V // 64 * 64)
    T = _spread(rng, 1, max(1, min(8192, LOGIT_BYTES // (V * SIZE[dtype]))))
    case = dict(op=op, T=T, V=V, dtype=dtype, temperature=rng.choice([0.6, 1.0, 1.0, 2.0]),
                masked=rng.random() < 0.3, pad=rng.choice([0, 0, -V % 128]))
    if T * (V + case["pad"]) * SIZE[dtype] > LOGIT_BYTES:
        case["pad"] = 0
    if op.startswith("distill"):
        case.update(K=_spread(rng, 1, 64 if case["masked"] else 256), ragged=rng.random() < 0.4)
    else:
        case.update(K=rng.choice([0, rng.randint(1, 32)]) if op == "logprob" else 0,
                    entropy=rng.random() < 0.6)
    return case


# ------------------------------------------------------------------------------------------ inputs


def _norm_inputs(case, seed):
    g = torch.Generator("cuda").manual_seed(seed)
    T, H, dt = case["T"], case["H"], DTYPES[case["dtype"]]
    wt = DTYPES[case["weights"]]
    wide = torch.randn((T, H + case["gap"]), generator=g, device="cuda")  # a slice of wider rows
    wide *= 0.5 + torch.rand((T, 1), generator=g, device="cuda")
    wide += 0.3 * torch.randn((T, 1), generator=g, device="cuda")
    i = dict(x=wide.to(dt)[:, :H])
    i["gamma"] = (1 + 0.2 * torch.randn(H, generator=g, device="cuda")).to(wt)
    i["beta"] = (0.2 * torch.randn(H, generator=g, device="cuda")).to(wt) if case["bias"] else None
    if case["op"] == "norm_grad":
        i["d_y"] = torch.randn((T, H), generator=g, device="cuda").to(dt)
    return i


def _logit_inputs(case, seed):
    g = torch.Generator("cuda").manual_seed(seed)
    T, V, K, dt = case["T"], case["V"], case["K"], DTYPES[case["dtype"]]
    z = torch.randn((T, V + case["pad"]), generator=g, device="cuda", dtype=dt)
    z *= (1.5 + 2.0 * torch.rand((T, 1), generator=g, device="cuda")).to(dt)
    z = z[:, :V]
    allowed = torch.arange(V, device="cuda")
    if case["masked"]:  # a grammar leaves a tenth of the vocabulary (never fewer than 64 tokens)
        order = torch.randperm(V, generator=g, device="cuda")
        keep = max(64, V // 10)
        allowed = order[:keep].sort().values
        z[:, order[keep:]] = -math.inf
    n = allowed.numel()
    i = dict(logits=z)
    if case["op"].startswith("logprob"):
        y = allowed[torch.randint(n, (T,), generator=g, device="cuda")]
        skip = torch.rand(T, generator=g, device="cuda") < 0.05  # padding tokens have no target
        i["targets"] = torch.where(skip, -100, y)
        i["d_logprob"] = torch.randn(T, generator=g, device="cuda")
        i["d_entropy"] = 0.1 * torch.randn(T, generator=g, device="cuda")
    else:
        base = torch.randint(n, (T, 1), generator=g, device="cuda")
        step = torch.randint(1, max(2, n // K), (T, 1), generator=g, device="cuda")
        i["index"] = allowed[(base + step * torch.arange(K, device="cuda")) % n]
        if case["ragged"]:
            short = torch.randint(1, K + 1, (T, 1), generator=g, device="cuda")
            i["index"] = torch.where(torch.arange(K, device="cuda") < short, i["index"], -1)
        t = 3 * torch.randn((T, K), generator=g, device="cuda")
        i["teacher"] = t.sort(dim=1, descending=True).values.to(dt)
        i["d_loss"] = torch.randn(T, generator=g, device="cuda")
    return i


def _norm_stats(x):
    v = x.float()
    mean = v.mean(1, keepdim=True)
    var = (v - mean).square().mean(1)
    return mean[:, 0], 1 / (var + EPS).sqrt()


def _row_stats(z, tau):
    v = z.float()
    m = v.amax(1)
    return torch.stack((m, ((v - m[:, None]) / tau).exp().sum(1)), 1)


def _teacher_weights(index, teacher, tau):
    t = (teacher.float() / tau).masked_fill(index < 0, -math.inf)
    e = (t - t.amax(1, keepdim=True)).exp()
    return e / e.sum(1, keepdim=True)


def _entropy(z, stats, tau):
    m, s = stats[:, :1], stats[:, 1:]
    d = (z.float() - m) / tau
    e = d.exp()
    return s[:, 0].log() - torch.where(e > 0, e * d, 0).sum(1) / s[:, 0]


def prepare(case, seed):
    op = case["op"]
    if op.startswith("norm"):
        i = _norm_inputs(case, seed)
        if op == "norm_grad":
            i["mean"], i["rstd"] = _norm_stats(i["x"])
    else:
        i = _logit_inputs(case, seed)
        tau = case["temperature"]
        if op == "logprob_grad":  # what the forward pass left
            i["stats"] = _row_stats(i["logits"], tau)
            i["entropy"] = _entropy(i["logits"], i["stats"], tau)
        if op == "distill_grad":
            i["stats"] = _row_stats(i["logits"], tau)
            i["weights"] = _teacher_weights(i["index"], i["teacher"], tau)
    return case, i


# --------------------------------------------------------------------------------------- one pass


def run(state):
    case, i = state
    return (_own if own else _plain)(case, i)


def _own(case, i):
    import mhc_hyper_connection_02_b200 as mhc
    op = case["op"]
    if op == "norm":
        return mhc.layer_norm(i["x"], i["gamma"], i["beta"], eps=EPS)
    if op == "norm_grad":
        return mhc.layer_norm_backward(i["d_y"], i["x"], i["gamma"], i["mean"], i["rstd"])
    tau = case["temperature"]
    if op == "logprob":
        out = mhc.token_logprobs(i["logits"], i["targets"], temperature=tau, top=case["K"],
                                 entropy=case["entropy"])
        return [o for o in out if o is not None]
    if op == "logprob_grad":
        ent = dict(d_entropy=i["d_entropy"], entropy=i["entropy"]) if case["entropy"] else {}
        return mhc.token_logprobs_backward(i["logits"], i["targets"], i["stats"], i["d_logprob"],
                                           temperature=tau, **ent)
    if op == "distill":
        return mhc.distill_topk(i["logits"], i["index"], i["teacher"], temperature=tau)
    return mhc.distill_topk_backward(i["logits"], i["index"], i["weights"], i["stats"], i["d_loss"],
                                     temperature=tau)


def _plain(case, i):
    op = case["op"]
    if op.startswith("norm"):
        x, gamma = i["x"].float(), i["gamma"].float()
        if op == "norm":
            mean, rstd = _norm_stats(i["x"])
            y = (x - mean[:, None]) * rstd[:, None] * gamma
            if i["beta"] is not None:
                y = y + i["beta"].float()
            return y.to(i["x"].dtype), mean, rstd
        dy, rstd = i["d_y"].float(), i["rstd"][:, None]
        xh = (x - i["mean"][:, None]) * rstd
        q = dy * gamma
        dx = rstd * (q - q.mean(1, keepdim=True) - xh * (q * xh).mean(1, keepdim=True))
        return dx.to(i["x"].dtype), (dy * xh).sum(0), dy.sum(0)
    tau = case["temperature"]
    z = i["logits"]
    V = z.shape[1]
    if op == "logprob":
        stats = _row_stats(z, tau)
        y = i["targets"]
        zy = z.gather(1, y.clamp(min=0)[:, None])[:, 0].float()
        lse = stats[:, 1].log()
        out = [torch.where(y >= 0, (zy - stats[:, 0]) / tau - lse, 0.0)]
        if case["entropy"]:
            out.append(_entropy(z, stats, tau))
        if case["K"]:
            # Keys that are unlike each other: the value's order, then the lower index first.
            b = z.float().contiguous().view(torch.int32)
            b = torch.where(b < 0, b ^ 0x7FFFFFFF, b).long()
            key = b * (1 << 32) + (V - 1 - torch.arange(V, device=z.device))
            top = V - 1 - (key.topk(case["K"], dim=1).values & 0xFFFFFFFF)
            zt = z.gather(1, top).float()
            out += [top, (zt - stats[:, :1]) / tau - lse[:, None]]
        return out + [stats]
    if op == "logprob_grad":
        m, s = i["stats"][:, :1], i["stats"][:, 1:]
        d = (z.float() - m) / tau
        p = d.exp() / s
        g = i["d_logprob"] * (i["targets"] >= 0)
        dz = -g[:, None] * p
        if case["entropy"]:
            lp = d - s.log()
            dz = dz - i["d_entropy"][:, None] * torch.where(p > 0, p * (lp + i["entropy"][:, None]), 0)
        dz.scatter_add_(1, i["targets"].clamp(min=0)[:, None], g[:, None])
        return (dz / tau).to(z.dtype)
    idx = i["index"]
    if op == "distill":
        stats = _row_stats(z, tau)
        w = _teacher_weights(idx, i["teacher"], tau)
        lp = (z.gather(1, idx.clamp(min=0)).float() - stats[:, :1]) / tau - stats[:, 1:].log()
        loss = torch.where(w > 0, w * (w.log() - lp), 0).sum(1)
        return loss, w, stats
    p = ((z.float() - i["stats"][:, :1]) / tau).exp() / i["stats"][:, 1:]
    p.scatter_add_(1, idx.clamp(min=0), -i["weights"])
    return (p * (i["d_loss"] / tau)[:, None]).to(z.dtype)


# ------------------------------------------------------------------------------- 64-bit definition


def _by_rows(f, T, V):
    step = max(1, (1 << 28) // V)
    parts = [f(slice(a, min(T, a + step))) for a in range(0, T, step)]
    return [torch.cat(c) if c[0] is not None else None for c in zip(*parts)]


def exact(case, seed):
    op = case["op"]
    if op.startswith("norm"):
        i = _norm_inputs(case, seed)
        x = i["x"].double()
        gamma = i["gamma"].double()
        sd = (x.var(1, unbiased=False, keepdim=True) + EPS).sqrt()
        hat = (x - x.mean(1, keepdim=True)) / sd
        if op == "norm":
            y = hat * gamma + (i["beta"].double() if i["beta"] is not None else 0)
            return y, x.mean(1), 1 / sd[:, 0]
        dy = i["d_y"].double()
        q = dy * gamma
        n = x.shape[1]
        # the projection of q off the row of ones and off hat, which has the squared norm n var / (var + eps)
        dx = (q - q.sum(1, keepdim=True) / n - hat * ((q * hat).sum(1, keepdim=True) / n)) / sd
        return dx, torch.einsum("th,th->h", dy, hat), dy.sum(0)
    i = _logit_inputs(case, seed)
    z, tau, V = i["logits"], case["temperature"], case["V"]
    if op == "logprob":
        def rows(r):
            v = z[r].double()
            lp = (v / tau).log_softmax(1)
            y = i["targets"][r]
            out = [lp.gather(1, y.clamp(min=0)[:, None])[:, 0].masked_fill(y < 0, 0)]
            if case["entropy"]:
                out.append(torch.special.entr(lp.exp()).sum(1))
            if case["K"]:
                order = v.sort(dim=1, descending=True, stable=True).indices[:, :case["K"]]
                out += [order, lp.gather(1, order)]
            top = v.amax(1, keepdim=True)
            return out + [torch.cat((top, ((v - top) / tau).exp().sum(1, keepdim=True)), 1)]
        return _by_rows(rows, case["T"], V)
    if op == "logprob_grad":
        def rows(r):
            lp = (z[r].double() / tau).log_softmax(1)
            p = lp.exp()
            y = i["targets"][r]
            g = torch.where(y >= 0, i["d_logprob"][r].double(), 0)
            one = torch.zeros_like(p).scatter_(1, y.clamp(min=0)[:, None], 1.0)
            dz = g[:, None] * (one - p)
            if case["entropy"]:
                ent = torch.special.entr(p)
                dz += i["d_entropy"][r].double()[:, None] * (ent - p * ent.sum(1, keepdim=True))
            return [dz / tau]
        return _by_rows(rows, case["T"], V)[0]
    w = i["teacher"].double().div(tau).masked_fill(i["index"] < 0, -math.inf).softmax(1)
    if op == "distill":
        def rows(r):
            v = z[r].double()
            lp = (v / tau).log_softmax(1).gather(1, i["index"][r].clamp(min=0))
            top = v.amax(1, keepdim=True)
            s = ((v - top) / tau).exp().sum(1, keepdim=True)
            loss = -(torch.special.entr(w[r]) + w[r] * lp).sum(1)
            return [loss, w[r], torch.cat((top, s), 1)]
        return _by_rows(rows, case["T"], V)

    def rows(r):
        p = (z[r].double() / tau).softmax(1)
        q = torch.zeros_like(p).scatter_add_(1, i["index"][r].clamp(min=0), w[r])
        return [(p - q) * (i["d_loss"][r].double() / tau)[:, None]]
    return _by_rows(rows, case["T"], V)[0]


def work(case):
    T, es = case["T"], SIZE[case["dtype"]]
    if case["op"].startswith("norm"):
        n = T * case["H"]
        ws = SIZE[case["weights"]] * case["H"]
        if case["op"] == "norm":
            return dict(bytes=2 * n * es + (2 if case["bias"] else 1) * ws + 8 * T, flops=7 * n)
        return dict(bytes=3 * n * es + ws + 8 * case["H"] + 8 * T, flops=14 * n)
    n, K = T * case["V"], case["K"]
    if case["op"] == "logprob":
        return dict(bytes=n * es + T * (8 + 4 + 8 + 4 * case["entropy"] + 12 * K),
                    flops=(6 if case["entropy"] else 4) * n)
    if case["op"] == "logprob_grad":
        return dict(bytes=2 * n * es + T * (8 + 4 + 8 + 8 * case["entropy"]),
                    flops=(6 if case["entropy"] else 4) * n)
    if case["op"] == "distill":
        return dict(bytes=n * es + T * (K * (8 + es + 4) + 4 + 8), flops=4 * n + 6 * T * K)
    return dict(bytes=2 * n * es + T * (K * 12 + 4 + 8), flops=4 * n + 2 * T * K)
