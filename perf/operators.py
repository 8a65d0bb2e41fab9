"""Workloads of the operators around the codec: the optimiser that makes a peer's pseudo-gradient (orthogonalised
momentum), the token log-probabilities that train a model and score an update, and the embedding table's lookup
and gradient.  Sizes are those of the 72B-class decoder layer (width 8192, key/value width 1024, MLP width 28,672,
vocabulary 262,208) and generic smaller or odd ones.

``run`` computes the plain form (elementary torch operations in 32 bits, rounded once at the end) or, with ``own``
true, calls the framework's operators."""
import math

import torch

own = False

COEFFICIENTS = (3.4445, -4.7750, 2.0315)
STEPS = 5
EPS = 1e-7
MU = 0.95

_DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16}


def listed():
    return [
        # one small matrix under the fused momentum step: latency of a chain of small products
        {"name": "orth_256x256_f32", "op": "orth", "batch": 1, "m": 256, "n": 256, "dtype": "f32", "momentum": True},
        # a stack of a small model's matrices, odd-sized, a view of a wider buffer, straight from bf16 gradients
        {"name": "orth_12x500x1000_bf16", "op": "orth", "batch": 12, "m": 500, "n": 1000, "dtype": "bf16", "momentum": False},
        # the decoder layer's k_proj / v_proj, fp32 gradient and momentum
        {"name": "orth_1024x8192_f32", "op": "orth", "batch": 1, "m": 1024, "n": 8192, "dtype": "f32", "momentum": True},
        # the decoder layer's gate_proj / up_proj (tall), the largest matrix product of a local step's optimiser
        {"name": "orth_28672x8192_bf16", "op": "orth", "batch": 1, "m": 28672, "n": 8192, "dtype": "bf16", "momentum": False},
        # one position while sampling from the model: the chosen token's probability and its alternatives
        {"name": "logp_1x262208_bf16", "op": "logp", "T": 1, "V": 262208, "dtype": "bf16", "top": 20},
        # scoring a sequence batch before and after an update is applied (a LossScore), with the top alternatives
        {"name": "logp_4096x262208_bf16", "op": "logp", "T": 4096, "V": 262208, "dtype": "bf16", "top": 5},
        # the loss gradient of a small model, odd vocabulary, fp32, with an entropy bonus
        {"name": "logp_grad_333x100003_f32", "op": "logp_grad", "T": 333, "V": 100003, "dtype": "f32", "entropy": True},
        # the loss gradient of a training micro-batch
        {"name": "logp_grad_4096x262208_bf16", "op": "logp_grad", "T": 4096, "V": 262208, "dtype": "bf16", "entropy": False},
        # the next tokens of a few sequences while sampling
        {"name": "embed_17x8192_bf16", "op": "embed", "T": 17, "D": 8192, "V": 262208, "dtype": "bf16"},
        # a training micro-batch's lookup
        {"name": "embed_16384x8192_f32", "op": "embed", "T": 16384, "D": 8192, "V": 65536, "dtype": "f32"},
        # the table gradient of a small model, odd width
        {"name": "embed_grad_2000x1001_f32", "op": "embed_grad", "T": 2000, "D": 1001, "V": 32768, "dtype": "f32"},
        # the table gradient of a training batch: common tokens repeat thousands of times, most rows get none
        {"name": "embed_grad_65536x8192_bf16", "op": "embed_grad", "T": 65536, "D": 8192, "V": 262208, "dtype": "bf16"},
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49)))))))


def draw(rng):
    op = rng.choice(["orth", "orth", "logp", "logp_grad", "embed", "embed_grad"])
    dtype = rng.choice(["f32", "bf16"])
    if op == "orth":
        m, n = _log_int(rng, 32, 8192), _log_int(rng, 32, 16384)
        batch = _log_int(rng, 1, 16) if m * n <= 1 << 21 else 1
        return {"op": op, "batch": batch, "m": m, "n": n, "dtype": dtype, "momentum": rng.random() < 0.5}
    if op in ("logp", "logp_grad"):
        c = {"op": op, "T": _log_int(rng, 1, 4096), "V": _log_int(rng, 500, 262208), "dtype": dtype}
        if c["T"] * c["V"] > 1 << 29:       # an fp32 case is no larger than the listed bf16 one
            c["T"] = (1 << 29) // c["V"]
        if op == "logp":
            c["top"] = rng.choice([0, 1, 5, 20, 32])
        else:
            c["entropy"] = rng.random() < 0.5
        return c
    c = {"op": op, "T": _log_int(rng, 1, 65536), "D": _log_int(rng, 64, 8192), "V": _log_int(rng, 500, 262208), "dtype": dtype}
    if op == "embed":
        c["T"] = max(1, min(c["T"], (1 << 27) // c["D"]))
    return c


def _generator(seed):
    return torch.Generator(device="cuda").manual_seed(int(seed))


def _matrix(b, m, n, gen):
    """A gradient-like matrix: a few strong directions over noise, rows of unlike scale."""
    rank = max(1, min(m, n) // 64)
    left = torch.randn(b, m, rank, generator=gen, device="cuda")
    right = torch.randn(b, rank, n, generator=gen, device="cuda")
    noise = torch.randn(b, m, n, generator=gen, device="cuda")
    rows = torch.exp(math.log(0.1) + torch.rand(b, m, 1, generator=gen, device="cuda") * math.log(100.0))
    return noise.mul_(rows).baddbmm_(left, right, alpha=2.0 / math.sqrt(rank)).mul_(2e-4)


def _token_ids(T, V, gen):
    """Token ids with a power-law frequency, as text has: the commonest few per cent of all, most ids never."""
    u = torch.rand(T, generator=gen, device="cuda", dtype=torch.float64)
    rank = (torch.exp(u * math.log(V + 1.0)) - 1.0).long().clamp_(0, V - 1)
    return (rank * 7919 + 13) % V if V % 7919 else rank


def prepare(case, seed):
    gen = _generator(seed)
    dt = _DTYPES[case["dtype"]]
    op = case["op"]
    if op == "orth":
        b, m, n = case["batch"], case["m"], case["n"]
        g = torch.empty(b, m, n + 8 if b > 1 else n, dtype=dt, device="cuda")[:, :, :n]
        for i in range(b):
            g[i] = _matrix(1, m, n, gen)[0]
        if b == 1:
            g = g[0]
        state = {"case": case, "grad": g, "momentum": None}
        if case["momentum"]:
            state["momentum"] = _matrix(b, m, n, gen).mul_(8.0).reshape(g.shape).contiguous()
        return state
    if op in ("logp", "logp_grad"):
        T, V = case["T"], case["V"]
        pad = -V % 8
        logits = torch.empty(T, V + pad, dtype=dt, device="cuda")[:, :V]
        bias = torch.log1p(torch.arange(V, device="cuda", dtype=torch.float32)).mul_(-0.7)
        targets = _token_ids(T, V, gen)
        for lo in range(0, T, 512):
            hi = min(T, lo + 512)
            z = torch.randn(hi - lo, V, generator=gen, device="cuda").mul_(2.0).add_(bias)
            sure = torch.rand(hi - lo, 1, generator=gen, device="cuda").mul_(14.0)
            z.scatter_add_(1, targets[lo:hi, None], sure)
            logits[lo:hi] = z
        masked = max(1, V // 50)            # entries a sampler or a padded vocabulary rules out
        logits[:, V - masked:] = -math.inf
        targets = targets.clamp(max=V - masked - 1)
        targets[torch.rand(T, generator=gen, device="cuda") < 0.05] = -100    # positions outside the loss
        state = {"case": case, "logits": logits, "targets": targets, "scale": 1.0 / 0.8}
        if op == "logp_grad":
            z = logits.float() * state["scale"]
            top = z.max(1, keepdim=True).values
            e = torch.exp(z - top)
            total = e.sum(1)
            state["lse"] = total.log() + top[:, 0]
            state["entropy"] = total.log() - (e * (z - top).clamp(min=-1e30)).sum(1) / total
            state["d_logp"] = torch.rand(T, generator=gen, device="cuda").add_(0.5).mul_(-1.0 / T)
            state["d_entropy"] = torch.randn(T, generator=gen, device="cuda").mul_(0.01 / T) if case["entropy"] else None
        return state
    T, D, V = case["T"], case["D"], case["V"]
    state = {"case": case, "ids": _token_ids(T, V, gen), "scale": math.sqrt(D)}
    if op == "embed":
        table = torch.empty(V, D, dtype=dt, device="cuda")
        for lo in range(0, V, 32768):
            hi = min(V, lo + 32768)
            table[lo:hi] = torch.randn(hi - lo, D, generator=gen, device="cuda").mul_(0.02)
        state["table"] = table
    else:
        state["grad"] = torch.randn(T, D, generator=gen, device="cuda").mul_(1e-3).to(dt)
    return state


# ---- the plain forms -----------------------------------------------------------------------------------------------

def _plain_orth(grad, momentum):
    g = grad.float()
    if momentum is not None:
        momentum.mul_(MU).add_(g)
        g = g + MU * momentum
    tall = g.shape[-2] > g.shape[-1]
    x = g.mT if tall else g
    x = x / ((x * x).sum((-2, -1), keepdim=True).sqrt() + EPS)
    a, b, c = COEFFICIENTS
    for _ in range(STEPS):
        gram = x @ x.mT
        x = a * x + (b * gram + c * (gram @ gram)) @ x
    x = (x.mT if tall else x).to(torch.bfloat16).contiguous()
    return {"out": x} if momentum is None else {"out": x, "momentum": momentum}


def _order_keys(logits):
    """Whole numbers that order raw logits from large to small, equal ones by index."""
    bits = (logits.float() + 0.0).view(torch.int32)
    ordered = torch.where(bits < 0, bits ^ 0x7FFFFFFF, bits).long()
    return (ordered << 32) | (0x7FFFFFFF - torch.arange(logits.shape[1], device=logits.device))


def _plain_logp(logits, targets, scale, top):
    z = logits.float() * scale
    peak = z.max(1, keepdim=True).values
    d = z - peak
    e = torch.exp(d)
    total = e.sum(1)
    log_total = total.log()
    lse = peak[:, 0] + log_total
    entropy = log_total - torch.where(e > 0, e * d, torch.zeros_like(d)).sum(1) / total
    chosen = d.gather(1, targets.clamp(min=0)[:, None])[:, 0] - log_total
    out = {"logp": torch.where(targets < 0, torch.zeros_like(chosen), chosen), "lse": lse, "entropy": entropy}
    if top:
        ids = torch.topk(_order_keys(logits), top, dim=1).indices
        out["top_ids"] = ids
        out["top_logp"] = d.gather(1, ids) - log_total[:, None]
    return out


def _plain_logp_grad(logits, targets, scale, lse, entropy, d_logp, d_entropy):
    d = logits.float() * scale - lse[:, None]
    p = torch.exp(d)
    w = torch.where(targets < 0, torch.zeros_like(d_logp), d_logp)
    g = p * -w[:, None]
    if d_entropy is not None:
        g = g - torch.where(p > 0, d_entropy[:, None] * p * (d + entropy[:, None]), torch.zeros_like(p))
    g.scatter_add_(1, targets.clamp(min=0)[:, None], w[:, None])
    return (g * scale).to(logits.dtype)


def _plain_embed_grad(ids, grad, rows, scale):
    return torch.zeros(rows, grad.shape[1], device=grad.device).index_add_(0, ids, grad.float()) * scale


def run(state):
    op = state["case"]["op"]
    if own:
        import compressed_pseudo_gradient_gb300 as spl
        if op == "orth":
            out = spl.orthogonalize(state["grad"], momentum=state["momentum"], mu=MU, steps=STEPS, coefficients=COEFFICIENTS, eps=EPS)
            return {"out": out} if state["momentum"] is None else {"out": out, "momentum": state["momentum"]}
        if op == "logp":
            r = spl.token_logprobs(state["logits"], state["targets"], scale=state["scale"], top=state["case"]["top"])
            out = {"logp": r.logp, "lse": r.lse, "entropy": r.entropy}
            if state["case"]["top"]:
                out["top_ids"], out["top_logp"] = r.top_ids, r.top_logp
            return out
        if op == "logp_grad":
            return spl.token_logprobs_grad(state["logits"], state["targets"], state["lse"], state["d_logp"], entropy=state["entropy"],
                                           d_entropy=state["d_entropy"], scale=state["scale"])
        if op == "embed":
            return spl.embedding(state["ids"], state["table"], scale=state["scale"])
        return spl.embedding_grad(state["ids"], state["grad"], state["case"]["V"], scale=state["scale"])
    if op == "orth":
        return _plain_orth(state["grad"], state["momentum"])
    if op == "logp":
        return _plain_logp(state["logits"], state["targets"], state["scale"], state["case"]["top"])
    if op == "logp_grad":
        return _plain_logp_grad(state["logits"], state["targets"], state["scale"], state["lse"], state["entropy"], state["d_logp"], state["d_entropy"])
    if op == "embed":
        return (state["table"][state["ids"]].float() * state["scale"]).to(state["table"].dtype)
    return _plain_embed_grad(state["ids"], state["grad"], state["case"]["V"], state["scale"])


# ---- the definitions in 64 bits ------------------------------------------------------------------------------------

def _exact_orth(case, state):
    m, n = sorted((case["m"], case["n"]))
    if case["batch"] * STEPS * (4.0 * m * m * n + 2.0 * m ** 3) > 6e12:
        return None
    u = state["grad"].double()
    new = None
    if state["momentum"] is not None:
        new = MU * state["momentum"].double() + u
        u = torch.add(u, new, alpha=MU)
    u = u.reshape(case["batch"], case["m"], case["n"])
    if case["m"] > case["n"]:
        u = u.transpose(1, 2)
    u = u / (u.pow(2).sum((1, 2), keepdim=True).sqrt() + EPS)
    a, b, c = COEFFICIENTS
    eye = torch.eye(u.shape[1], dtype=torch.float64, device=u.device)
    for _ in range(STEPS):
        s = torch.bmm(u, u.transpose(1, 2))
        u = torch.bmm(a * eye + torch.bmm(s, b * eye + c * s), u)
    if case["m"] > case["n"]:
        u = u.transpose(1, 2)
    u = u.reshape(state["grad"].shape).contiguous()
    return {"out": u} if new is None else {"out": u, "momentum": new}


def exact(case, seed):
    state = prepare(case, seed)
    op = case["op"]
    if op == "orth":
        return _exact_orth(case, state)
    if op == "logp":
        rows = []
        for lo in range(0, case["T"], 256):
            z = state["logits"][lo:lo + 256].double() * state["scale"]
            t = state["targets"][lo:lo + 256]
            logq = z - torch.logsumexp(z, 1, keepdim=True)
            picked = logq.gather(1, t.clamp(min=0)[:, None])[:, 0] * (t >= 0)
            entropy = -(torch.exp(logq) * logq.masked_fill(logq == -math.inf, 0.0)).sum(1)
            part = [picked, torch.logsumexp(z, 1), entropy]
            if case["top"]:
                part += [logq.sort(dim=1, descending=True, stable=True).values[:, :case["top"]]]
            rows.append(part)
        cat = [torch.cat(x) for x in zip(*rows)]
        out = {"logp": cat[0], "lse": cat[1], "entropy": cat[2]}
        if case["top"]:
            out["top_ids"], out["top_logp"] = None, cat[3]
        return out
    if op == "logp_grad":
        T, V = case["T"], case["V"]
        out = torch.empty(T, V, dtype=torch.float64, device="cuda")
        for lo in range(0, T, 256):
            z = state["logits"][lo:lo + 256].double() * state["scale"]
            t = state["targets"][lo:lo + 256]
            logq = z - state["lse"][lo:lo + 256, None].double()
            q = torch.exp(logq)
            w = state["d_logp"][lo:lo + 256].double() * (t >= 0)
            hot = torch.zeros_like(q).scatter_(1, t.clamp(min=0)[:, None], 1.0)
            g = w[:, None] * (hot - q)
            if state["d_entropy"] is not None:
                h = state["entropy"][lo:lo + 256, None].double()
                g -= state["d_entropy"][lo:lo + 256, None].double() * q * (logq.masked_fill(q == 0, 0.0) + h)
            out[lo:lo + 256] = g * state["scale"]
        return out
    if op == "embed":
        return torch.index_select(state["table"], 0, state["ids"]).double().mul_(state["scale"])
    order = torch.argsort(state["ids"], stable=True)
    ids = state["ids"][order]
    last = torch.ones_like(ids, dtype=torch.bool)
    last[:-1] = ids[1:] != ids[:-1]
    ends = last.nonzero()[:, 0]
    out = torch.zeros(case["V"], case["D"], dtype=torch.float64, device="cuda")
    for lo in range(0, case["D"], 1024):
        running = state["grad"][:, lo:lo + 1024][order].double().cumsum(0)[ends]
        running[1:] -= running[:-1].clone()
        out[ids[ends], lo:lo + 1024] = running * state["scale"]
    return out


def work(case):
    size = 4 if case["dtype"] == "f32" else 2
    op = case["op"]
    if op == "orth":
        b, (m, n) = case["batch"], sorted((case["m"], case["n"]))
        moved = b * m * n * (size + 2 + (8 if case["momentum"] else 0))
        # the two symmetric products count one triangle
        return {"bytes": moved, "flops": b * STEPS * (3.0 * m * m * n + m ** 3)}
    if op == "logp":
        T, V = case["T"], case["V"]
        return {"bytes": T * (V * size + 8 + 12 + 12 * case["top"]), "flops": 6.0 * T * V}
    if op == "logp_grad":
        T, V = case["T"], case["V"]
        return {"bytes": T * (2 * V * size + 8 + 12), "flops": 6.0 * T * V}
    T, D, V = case["T"], case["D"], case["V"]
    if op == "embed":
        return {"bytes": T * (2 * D * size + 8), "flops": float(T * D)}
    return {"bytes": T * (D * size + 8) + V * D * 4, "flops": 2.0 * T * D}
