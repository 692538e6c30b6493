"""Timed cases of the operators that stand between the QLoRA linears of a
training step and at its end, each with a plain torch form and an exact form
in 64 bits:

  norm        layer norm and root-mean-square norm, forward and backward with
              the weight's and the bias's gradients
  epilogue    the linear layer with bias, activation and residual: on the NF4
              weight with adapters (with the backward through the activation)
              and on a merged 4-bit weight
  preference  the loss on paired log ratios of packed sequences, and dlogits
  distill     distillation from a teacher's top logits: loss and dlogits

``own`` False computes the plain form, True calls the library.
"""

import math

import torch

own = False

DEV = "cuda"

# the sixteen NF4 values, ascending
NF4 = (-1.0, -0.6961928009986877, -0.5250730514526367, -0.39491748809814453, -0.28444138169288635,
       -0.18477343022833334, -0.09105003625154495, 0.0, 0.07958029955625534, 0.16093020141124725,
       0.24611230194568634, 0.33791524171829224, 0.44070982933044434, 0.5626170039176941, 0.7229568362236023, 1.0)

IGNORE = -100


# ---------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------
def listed():
    return [
        # one token through the norm before a 7B attention block: latency
        {"name": "rms T1 C4096 fwd", "op": "norm", "T": 1, "C": 4096, "rms": True, "f32": False, "wf32": False,
         "bwd": False},
        # one training sequence of odd length, weights kept in fp32
        {"name": "layer T1001 C4096 fwd+bwd", "op": "norm", "T": 1001, "C": 4096, "rms": False, "f32": False,
         "wf32": True, "bwd": True},
        # a training batch at the 65B hidden size
        {"name": "rms T16384 C8192 fwd+bwd", "op": "norm", "T": 16384, "C": 8192, "rms": True, "f32": False,
         "wf32": False, "bwd": True},
        # decode of one token: 7B output projection onto the residual stream
        {"name": "nf4 T1 4096x4096 r16 bias res", "op": "epilogue", "T": 1, "N": 4096, "K": 4096, "r": 16, "group": 0,
         "act": "none", "bias": True, "res": True, "bwd": False},
        # 7B-shaped first MLP linear with bias and activation in training
        {"name": "nf4 T1000 11008x4096 r16 gelu fwd+bwd", "op": "epilogue", "T": 1000, "N": 11008, "K": 4096, "r": 16,
         "group": 0, "act": "gelu", "bias": True, "res": False, "bwd": True},
        # decode batch on a merged weight: down projection onto the residual stream
        {"name": "q4g T24 4096x11008 g128 bias res", "op": "epilogue", "T": 24, "N": 4096, "K": 11008, "r": 0,
         "group": 128, "act": "none", "bias": True, "res": True, "bwd": False},
        # one pair of short answers
        {"name": "pref 1 pair 16 tok V32000", "op": "preference", "pairs": 1, "T": 16, "V": 32000, "f32": False,
         "kind": "sigmoid", "average": False, "prompt": 0.0},
        # a batch of pairs with their prompts masked
        {"name": "pref 4 pairs 3500 tok V32000", "op": "preference", "pairs": 4, "T": 3500, "V": 32000, "f32": False,
         "kind": "sigmoid", "average": False, "prompt": 0.3},
        # an odd vocabulary, fp32 logits, length-normalised
        {"name": "pref 8 pairs 6001 tok V50257 f32", "op": "preference", "pairs": 8, "T": 6001, "V": 50257,
         "f32": True, "kind": "squared", "average": True, "prompt": 0.5},
        # the last token of a prompt
        {"name": "distill T1 V32000 K8", "op": "distill", "T": 1, "V": 32000, "K": 8, "f32": False, "tau": 1.0,
         "alpha": 0.0},
        # one training batch, softened targets
        {"name": "distill T2048 V32000 K64", "op": "distill", "T": 2048, "V": 32000, "K": 64, "f32": False,
         "tau": 2.0, "alpha": 0.0},
        # a large vocabulary, mixed with the labels' cross entropy
        {"name": "distill T4000 V128000 K32 ce", "op": "distill", "T": 4000, "V": 128000, "K": 32, "f32": False,
         "tau": 1.0, "alpha": 0.5},
    ]


def _log(rng, lo, hi):
    """An integer in [lo, hi], its logarithm uniform."""
    return min(hi, max(lo, int(round(lo * (hi / lo) ** rng.random()))))


def draw(rng):
    op = rng.choice(["norm", "epilogue", "preference", "distill"])
    if op == "norm":
        f32 = rng.random() < 0.3
        return {"op": op, "T": _log(rng, 1, 8192 if f32 else 16384), "C": 8 * _log(rng, 1, 1024),
                "rms": rng.random() < 0.5, "f32": f32, "wf32": rng.random() < 0.5, "bwd": rng.random() < 0.7}
    if op == "epilogue":
        act = rng.choice(["none", "silu", "gelu", "gelu_tanh"])
        c = {"op": op, "act": act, "bias": rng.random() < 0.6, "res": rng.random() < 0.5}
        if rng.random() < 0.4:
            c.update(T=_log(rng, 1, 64), N=8 * _log(rng, 1, 1376), K=8 * _log(rng, 4, 1376), r=0,
                     group=rng.choice([32, 64, 128]), bwd=False)
        else:
            c.update(T=_log(rng, 1, 1000), N=8 * _log(rng, 1, 1376), K=64 * _log(rng, 1, 64),
                     r=rng.choice([0, 3, 8, 16, 33, 64]), group=0, bwd=rng.random() < 0.5)
        return c
    f32 = rng.random() < 0.3
    if op == "preference":
        pairs = _log(rng, 1, 16)
        return {"op": op, "pairs": pairs, "T": _log(rng, 2 * pairs, 4096), "V": _log(rng, 300, 50257), "f32": f32,
                "kind": rng.choice(["sigmoid", "hinge", "squared"]), "average": rng.random() < 0.4,
                "prompt": rng.choice([0.0, 0.3, 0.6])}
    V = _log(rng, 300, 128000)
    return {"op": op, "T": _log(rng, 1, max(1, min(8192, 250000000 // V))), "V": V, "K": _log(rng, 1, 128), "f32": f32,
            "tau": rng.choice([1.0, 1.0, 2.0, 0.7]), "alpha": rng.choice([0.0, 0.0, 0.1, 0.5])}


def work(case):
    op = case["op"]
    if op == "norm":
        n = case["T"] * case["C"]
        e, w = (4 if case["f32"] else 2), (4 if case["wf32"] else 2)
        nw = 1 if case["rms"] else 2
        b, f = 2 * e * n + w * nw * case["C"], 8 * n
        if case["bwd"]:  # x stays an input of the pass, read once
            b += 2 * e * n + 4 * nw * case["C"]
            f += 14 * n
        return {"bytes": b, "flops": f}
    if op == "epilogue":
        T, N, K, r = case["T"], case["N"], case["K"], case["r"]
        b = 2 * T * K + 2 * T * N + (2 * N if case["bias"] else 0) + (2 * T * N if case["res"] else 0)
        f = 2 * T * N * K + 2 * T * r * (N + K) + (12 * T * N if case["act"] != "none" else 0)
        b += N * K * (0.5 + 1 / 64) + 2 * r * (N + K) if case["group"] == 0 else \
            N * K / 2 + 3 * N * -(-K // case["group"])
        if case["bwd"]:  # dY in, dZ out
            b += 4 * T * N + (4 * N if case["bias"] else 0)
            f += 12 * T * N
        return {"bytes": b, "flops": f}
    e = 4 if case["f32"] else 2
    if op == "preference":  # masked rows are not read, their gradient rows are written
        n = case["T"] * case["V"]
        return {"bytes": e * n * (1 - case["prompt"]) + e * n, "flops": 8 * n * (1 - case["prompt"])}
    n = case["T"] * case["V"]
    return {"bytes": 2 * e * n + case["T"] * (case["K"] * 12 + 12), "flops": (8 if case["alpha"] == 0 else 11) * n}


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------
def _randn(gen, *shape):
    return torch.randn(*shape, generator=gen, device=DEV)


def _activation(gen, T, K):
    """Activations with a few large channels, as transformer layers have."""
    x = _randn(gen, T, K)
    big = torch.rand(K, generator=gen, device=DEV) < 0.005
    return torch.where(big, 20 * x, x)


def _nf4_weight(gen, N, K):
    """A frozen NF4 weight with double-quantized constants, W ~ 0.02 N(0, 1)."""
    w = (0.02 * _randn(gen, N, K)).view(-1, 64)
    a = w.abs().amax(dim=1)
    t = torch.tensor(NF4, device=DEV)
    c = torch.bucketize(w / a[:, None], (t[1:] + t[:-1]) / 2).to(torch.uint8).view(-1, 2)
    mean = a.double().mean().float()
    d = a - mean
    n = d.numel()
    pad = torch.nn.functional.pad(d, (0, -n % 256)).view(-1, 256)
    scale = pad.abs().amax(dim=1) / 448
    c8 = (pad / scale.clamp(min=1e-30)[:, None]).to(torch.float8_e4m3fn).view(-1)[:n].contiguous()
    return {"packed": (c[:, 0] * 16 + c[:, 1]).contiguous(), "c8": c8.view(torch.uint8),
            "dq_scale": scale.contiguous(), "dq_mean": mean.view(1)}


def _q4g_weight(gen, N, K, group):
    """A 4-bit weight with bf16 scales and zero points per group of a row."""
    g = -(-K // group)
    q = torch.randint(0, 16, (N, -(-K // 32) * 32), generator=gen, device=DEV, dtype=torch.int32)
    return {"packed": (q[:, 0::2] * 16 + q[:, 1::2]).to(torch.uint8),
            "wscale": (0.004 * (0.5 + torch.rand(N, g, generator=gen, device=DEV))).to(torch.bfloat16),
            "zero": torch.randint(5, 11, (N, g), generator=gen, device=DEV, dtype=torch.int32).to(torch.uint8)}


def _logits(gen, T, V, f32, labels):
    """Logits that favour the label by a few units, as a trained model's do."""
    z = 2.5 * _randn(gen, T, V)
    z[torch.arange(T, device=DEV), labels] += 5.0
    return z if f32 else z.to(torch.bfloat16)


def _log_softmax_rows(z, labels):
    """log softmax of each row at its label, fp64, a few rows at a time."""
    out = []
    for zi, li in zip(z.split(256), labels.split(256)):
        zi = zi.double()
        m = zi.amax(dim=1)
        out.append(zi.gather(1, li[:, None])[:, 0] - m - torch.log(torch.exp(zi - m[:, None]).sum(dim=1)))
    return torch.cat(out)


def _sequence_sums(v, start):
    """Sums of v (fp64 [T]) over the rows of each sequence."""
    c = torch.cat([torch.zeros(1, dtype=torch.float64, device=v.device), torch.cumsum(v, 0)])
    return c[start[1:]] - c[start[:-1]]


def prepare(case, seed):
    gen = torch.Generator(device=DEV)
    gen.manual_seed(int(seed))
    s = dict(case)
    op = case["op"]
    if op == "norm":
        T, C = case["T"], case["C"]
        dt, wt = (torch.float32 if case[k] else torch.bfloat16 for k in ("f32", "wf32"))
        s["X"] = (_activation(gen, T, C) + 0.2).to(dt)
        s["w"] = (1 + 0.1 * _randn(gen, C)).to(wt)
        s["b"] = None if case["rms"] else (0.1 * _randn(gen, C)).to(wt)
        s["dY"] = _randn(gen, T, C).to(dt)
        s["eps"] = 1e-5
    elif op == "epilogue":
        T, N, K, r = case["T"], case["N"], case["K"], case["r"]
        s["X"] = _activation(gen, T, K).to(torch.bfloat16)
        s["b"] = (0.5 * _randn(gen, N)).to(torch.bfloat16) if case["bias"] else None
        s["R"] = _randn(gen, T, N).to(torch.bfloat16) if case["res"] else None
        s["dY"] = _randn(gen, T, N).to(torch.bfloat16) if case["bwd"] else None
        s["A"] = s["B"] = None
        s["scale"] = 1.0
        if case["group"]:
            s.update(_q4g_weight(gen, N, K, case["group"]))
        else:
            s.update(_nf4_weight(gen, N, K))
            if r > 0:
                s["A"] = (_randn(gen, r, K) / 64).to(torch.bfloat16)
                s["B"] = (0.05 * _randn(gen, N, r)).to(torch.bfloat16)
                s["scale"] = 16.0 / r
    else:
        T, V = case["T"], case["V"]
        labels = torch.randint(0, V, (T,), generator=gen, device=DEV)
        s["logits"] = _logits(gen, T, V, case["f32"], labels)
        if op == "preference":
            P = case["pairs"]
            # 2 P sequences of unequal lengths, one row at least each
            cuts = torch.randperm(T - 1, generator=gen, device=DEV)[: 2 * P - 1].sort().values + 1
            ends = torch.tensor([0, T], device=DEV)
            s["start"] = torch.cat([ends[:1], cuts, ends[1:]])
            at = torch.arange(T, device=DEV)
            seq = torch.searchsorted(s["start"], at, right=True) - 1
            first, last = s["start"][seq], s["start"][seq + 1]
            prompt = at < first + (case["prompt"] * (last - first)).long()
            lp = torch.where(prompt, 0.0, _log_softmax_rows(s["logits"], labels))
            ref = _sequence_sums(lp, s["start"])
            if case["average"]:
                ref = ref / _sequence_sums((~prompt).double(), s["start"])
            s["ref"] = (ref + 3 * _randn(gen, 2 * P)).float()
            s["labels"] = torch.where(prompt, IGNORE, labels)
            s["beta"], s["smooth"] = 0.1, (0.1 if case["kind"] == "sigmoid" else 0.0)
            s["dloss"] = (0.5 + torch.rand(P, generator=gen, device=DEV)) / P
        else:
            K = case["K"]
            # the teacher agrees with the student in part: its top tokens are the label and random others
            at = torch.randint(0, V, (T, K), generator=gen, device=DEV)
            at[:, 0] = labels
            s["index"] = at
            s["top"] = (2 * _randn(gen, T, K)).sort(dim=1, descending=True).values
            s["labels"] = labels if case["alpha"] > 0 else None
            s["weight"] = torch.full((T,), 1.0 / T, device=DEV)
    if own and op == "epilogue":  # the handle around these tensors that a program keeps with them
        import bit_nf4_quantized_16_amd as qn
        if case["group"]:
            s["w"] = qn.Q4GWeight(case["N"], case["K"], case["group"], s["packed"], s["wscale"], s["zero"])
        else:
            s["w"] = qn.NF4Weight(case["N"], case["K"], s["packed"], c8=s["c8"], dq_scale=s["dq_scale"],
                                  dq_mean=s["dq_mean"])
    return s


# ---------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------
def run(s):
    return _run_own(s) if own else _run_plain(s)


def _run_own(s):
    import bit_nf4_quantized_16_amd as qn

    op = s["op"]
    if op == "norm":
        Y, mean, rstd = qn.norm_fwd(s["X"], s["w"], s["b"], eps=s["eps"], rms=s["rms"], stats=s["bwd"])
        if not s["bwd"]:
            return Y
        dX, dW, dB = qn.norm_bwd(s["X"], s["w"], s["dY"], mean, rstd, need_db=not s["rms"])
        return (Y, dX, dW) if s["rms"] else (Y, dX, dW, dB)
    if op == "epilogue":
        if s["group"]:
            return qn.q4g_linear_fwd_epilogue(s["w"], s["X"], bias=s["b"], act=s["act"], residual=s["R"])
        Y, U, Z = qn.qlora_linear_fwd_epilogue(s["w"], s["X"], s["A"], s["B"], s["scale"], bias=s["b"], act=s["act"],
                                               residual=s["R"], save_u=s["bwd"], save_z=s["bwd"])
        if not s["bwd"]:
            return Y
        dZ, db = qn.epilogue_bwd(s["dY"], Z, act=s["act"], need_dbias=s["bias"])
        return {"Y": Y, "dZ": dZ, "db": db} if s["bias"] else {"Y": Y, "dZ": dZ}
    if op == "preference":
        loss, logp, state = qn.preference_loss_fwd(s["logits"], s["labels"], s["start"], s["ref"], beta=s["beta"],
                                                   label_smoothing=s["smooth"], kind=s["kind"], average=s["average"])
        return loss, logp, qn.preference_loss_bwd(s["logits"], s["labels"], state, s["dloss"])
    return qn.distill_loss(s["logits"], s["index"], s["top"], labels=s["labels"], temperature=s["tau"],
                           alpha=s["alpha"], weight=s["weight"], need_grad=True)


def _nf4_expand(s):
    """W' as fp32 values, rounded to bf16 once (the weight the layer multiplies with)."""
    p = s["packed"]
    c = torch.stack([p >> 4, p & 15], dim=1).view(-1, 64).long()
    e = s["c8"].view(torch.float8_e4m3fn).float().view(-1)
    a = e * s["dq_scale"].repeat_interleave(256)[: e.numel()] + s["dq_mean"]
    return (torch.tensor(NF4, device=DEV)[c] * a[:, None]).to(torch.bfloat16).float().view(s["N"], s["K"])


def _q4g_expand(s):
    """W' fp32 [N, K] = s (q - z)."""
    p, group, K = s["packed"], s["group"], s["K"]
    q = torch.stack([p >> 4, p & 15], dim=2).view(p.shape[0], -1)[:, :K].float()
    at = torch.arange(K, device=p.device) // group
    return (q - s["zero"].float()[:, at]) * s["wscale"].float()[:, at]


def _erf_cdf(z):
    """The normal distribution function: from erfc's side where it is small."""
    return 0.5 * torch.erfc(z * -math.sqrt(0.5))


def _act(z, act):
    if act == "silu":
        return z / (1 + torch.exp(-z))
    if act == "gelu":
        return z * _erf_cdf(z)
    if act == "gelu_tanh":
        return z / (1 + torch.exp(-2 * math.sqrt(2 / math.pi) * (z + 0.044715 * z * z * z)))
    return z


def _act_slope(z, act):
    if act == "silu":
        p = 1 / (1 + torch.exp(-z))
        return p * (1 + z * (1 - p))
    if act == "gelu":
        return _erf_cdf(z) + z * torch.exp(-0.5 * z * z) / math.sqrt(2 * math.pi)
    if act == "gelu_tanh":
        c = 2 * math.sqrt(2 / math.pi)
        p = 1 / (1 + torch.exp(-c * (z + 0.044715 * z * z * z)))
        return p + z * p * (1 - p) * c * (1 + 3 * 0.044715 * z * z)
    return torch.ones_like(z)


def _run_plain(s):
    op = s["op"]
    if op == "norm":
        x, w = s["X"].float(), s["w"].float()
        c = x if s["rms"] else x - x.mean(dim=1, keepdim=True)
        r = 1 / torch.sqrt((c * c).mean(dim=1, keepdim=True) + s["eps"])
        h = c * r
        y = (h * w if s["b"] is None else h * w + s["b"].float()).to(s["X"].dtype)
        if not s["bwd"]:
            return y
        d = s["dY"].float()
        g = d * w
        t = g - h * (g * h).mean(dim=1, keepdim=True)
        if not s["rms"]:
            t = t - g.mean(dim=1, keepdim=True)
        dx, dw = (t * r).to(s["X"].dtype), (d * h).double().sum(dim=0).float()
        return (y, dx, dw) if s["rms"] else (y, dx, dw, d.double().sum(dim=0).float())
    if op == "epilogue":
        x = s["X"].float()
        z = x @ (_q4g_expand(s) if s["group"] else _nf4_expand(s)).T
        if s["r"] > 0:
            z = z + s["scale"] * ((x @ s["A"].float().T) @ s["B"].float().T)
        if s["b"] is not None:
            z = z + s["b"].float()
        y = _act(z, s["act"])
        y = (y if s["R"] is None else y + s["R"].float()).to(torch.bfloat16)
        if not s["bwd"]:
            return y
        dz = s["dY"].float() * _act_slope(z, s["act"])
        out = {"Y": y, "dZ": dz.to(torch.bfloat16)}
        if s["bias"]:
            out["db"] = dz.double().sum(dim=0).float()
        return out
    z = s["logits"].float()
    rows = torch.arange(z.shape[0], device=z.device)
    if op == "preference":
        m = z.amax(dim=1, keepdim=True)
        e = torch.exp(z - m)
        total = e.sum(dim=1, keepdim=True)
        on = s["labels"] != IGNORE
        at = torch.where(on, s["labels"], 0)
        lp = torch.where(on, z[rows, at] - (m + torch.log(total))[:, 0], 0.0)
        sums = _sequence_sums(lp.double(), s["start"])
        per = torch.ones_like(sums)
        if s["average"]:
            per = 1 / _sequence_sums(on.double(), s["start"]).clamp(min=1)
            sums = sums * per
        d = sums - s["ref"].double()
        d = d[0::2] - d[1::2]
        x = s["beta"] * d
        if s["kind"] == "sigmoid":
            p = 1 / (1 + torch.exp(x))  # of -x
            loss = -(1 - s["smooth"]) * torch.log(1 - p) - s["smooth"] * torch.log(p)
            slope = s["beta"] * (s["smooth"] * (1 - p) - (1 - s["smooth"]) * p)
        elif s["kind"] == "hinge":
            loss = (1 - x).clamp(min=0)
            slope = torch.where(x < 1, -s["beta"], 0.0).double()
        else:
            loss = (d - 0.5 / s["beta"]) ** 2
            slope = 2 * (d - 0.5 / s["beta"])
        slope = torch.stack([slope, -slope], dim=1).view(-1) * s["dloss"].double().repeat_interleave(2) * per
        seq = torch.searchsorted(s["start"], rows, right=True) - 1
        f = torch.where(on, slope[seq].float(), 0.0)
        dz = e / total * -f[:, None]
        dz[rows, at] += f
        return loss.float(), sums.float(), dz.to(s["logits"].dtype)
    tau, alpha = s["tau"], s["alpha"]
    k = s["index"]
    t = s["top"].float() / tau
    t = t - t.amax(dim=1, keepdim=True)
    p = torch.exp(t)
    p = p / p.sum(dim=1, keepdim=True)
    m = z.amax(dim=1, keepdim=True)
    e = torch.exp((z - m) / tau)
    total = e.sum(dim=1, keepdim=True)
    logq = (z.gather(1, k) - m) / tau - torch.log(total)
    loss = (1 - alpha) * tau * tau * (p * (torch.log(p) - logq)).sum(dim=1)
    dz = (1 - alpha) * tau * (e / total)
    dz.scatter_add_(1, k, -(1 - alpha) * tau * p)
    if alpha > 0:
        if tau != 1.0:
            e = torch.exp(z - m)
            total = e.sum(dim=1, keepdim=True)
        at = s["labels"]
        loss = loss - alpha * ((z[rows, at] - m[:, 0]) - torch.log(total)[:, 0])
        dz = dz + alpha * (e / total)
        dz[rows, at] -= alpha
    return loss, (dz * s["weight"][:, None]).to(s["logits"].dtype)


# ---------------------------------------------------------------------------
# the definitions in 64 bits
# ---------------------------------------------------------------------------
def _exact_weight(s):
    """W' [N, K] in fp64: the stored codes and constants, rounded as each
    weight's definition says."""
    K = s["K"]
    j = torch.arange(K, device=DEV)
    if s["group"]:
        q = torch.where(j % 2 == 0, s["packed"][:, j // 2] >> 4, s["packed"][:, j // 2] & 15).double()
        at = j // s["group"]
        return s["wscale"].double()[:, at] * (q - s["zero"].double()[:, at])
    packed = s["packed"].view(s["N"], K // 2)
    c = torch.where(j % 2 == 0, packed[:, j // 2] >> 4, packed[:, j // 2] & 15).long()
    b = s["c8"].int()
    ex, fr = (b >> 3) & 15, (b & 7).double()
    e = torch.where(ex == 0, fr / 512, torch.ldexp(1 + fr / 8, ex - 7)) * torch.where(b >= 128, -1.0, 1.0)
    group = torch.arange(e.numel(), device=DEV) // 256
    a = ((e * s["dq_scale"].double()[group]).float().double() + s["dq_mean"].double()).float().double()
    w = torch.tensor(NF4, device=DEV).double()[c] * a.view(s["N"], K // 64)[:, j // 64]
    return w.float().to(torch.bfloat16).double()


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "norm":
        x, w = s["X"].double(), s["w"].double()
        n = case["C"]
        mean = torch.zeros_like(x[:, :1]) if case["rms"] else x.sum(dim=1, keepdim=True) / n
        r = torch.rsqrt(((x - mean) ** 2).sum(dim=1, keepdim=True) / n + s["eps"])
        h = (x - mean) * r
        y = h * w + (0 if s["b"] is None else s["b"].double())
        if not case["bwd"]:
            return y
        d = s["dY"].double()
        g = d * w
        dx = r * (g - h * (g * h).sum(dim=1, keepdim=True) / n)
        if case["rms"]:
            return y, dx, (d * h).sum(dim=0)
        return y, dx - r * g.sum(dim=1, keepdim=True) / n, (d * h).sum(dim=0), d.sum(dim=0)
    if op == "epilogue":
        x = s["X"].double()
        z = torch.mm(x, _exact_weight(s).T.contiguous())
        if case["r"] > 0:
            u = torch.mm(x, s["A"].double().T.contiguous())
            z = torch.addmm(z, u, s["B"].double().T.contiguous(), alpha=s["scale"])
        if case["bias"]:
            z = z + s["b"].double()
        act = case["act"]
        c = 2 * math.sqrt(2 / math.pi)
        if act == "none":
            y, slope = z, torch.ones_like(z)
        elif act == "gelu":
            cdf = torch.special.ndtr(z)
            y, slope = z * cdf, cdf + z * torch.exp(-z * z / 2) / math.sqrt(2 * math.pi)
        else:
            u, du = (z, torch.ones_like(z)) if act == "silu" else (c * (z + 0.044715 * z ** 3),
                                                                  c * (1 + 0.134145 * z * z))
            p = torch.sigmoid(u)
            y, slope = z * p, p + z * p * torch.sigmoid(-u) * du
        if case["res"]:
            y = y + s["R"].double()
        if not case["bwd"]:
            return y
        dz = s["dY"].double() * slope
        return {"Y": y, "dZ": dz, "db": dz.sum(dim=0)} if case["bias"] else {"Y": y, "dZ": dz}
    T, V = case["T"], case["V"]
    if op == "preference":
        live = (s["labels"] >= 0).nonzero()[:, 0]
        start = s["start"].tolist()
        labels = s["labels"]
        lp = torch.zeros(T, dtype=torch.float64, device=DEV)
        for rows in live.split(512):
            q = torch.log_softmax(s["logits"][rows].double(), dim=1)
            lp[rows] = q[torch.arange(rows.numel(), device=DEV), labels[rows]]
        sums, count = [], []
        for a, b in zip(start[:-1], start[1:]):
            n = int((labels[a:b] >= 0).sum())
            count.append(max(n, 1) if case["average"] else 1)
            sums.append(lp[a:b].sum() / count[-1])
        sums = torch.stack(sums)
        d = (sums - s["ref"].double()).view(-1, 2)
        d = (d[:, 0] - d[:, 1]).requires_grad_()
        x = s["beta"] * d
        if case["kind"] == "sigmoid":
            loss = -(1 - s["smooth"]) * torch.nn.functional.logsigmoid(x) \
                - s["smooth"] * torch.nn.functional.logsigmoid(-x)
        elif case["kind"] == "hinge":
            loss = torch.relu(1 - x)
        else:
            loss = (d - 1 / (2 * s["beta"])) ** 2
        slope, = torch.autograd.grad((loss * s["dloss"].double()).sum(), d)
        f = torch.zeros(T, dtype=torch.float64, device=DEV)
        for i, (a, b) in enumerate(zip(start[:-1], start[1:])):
            f[a:b] = slope[i // 2] * (1 if i % 2 == 0 else -1) / count[i]
        dz = torch.zeros(T, V, dtype=torch.float64, device=DEV)
        for rows in live.split(512):
            g = -torch.softmax(s["logits"][rows].double(), dim=1)
            g[torch.arange(rows.numel(), device=DEV), labels[rows]] += 1
            dz[rows] = g * f[rows][:, None]
        return loss.detach(), sums, dz
    tau, alpha = case["tau"], case["alpha"]
    loss = torch.empty(T, dtype=torch.float64, device=DEV)
    dz = torch.empty(T, V, dtype=torch.float64, device=DEV)
    for rows in torch.arange(T, device=DEV).split(512):
        z = s["logits"][rows].double()
        at = s["index"][rows]
        logp = torch.log_softmax(s["top"][rows].double() / tau, dim=1)
        logq = torch.log_softmax(z / tau, dim=1)
        loss[rows] = (1 - alpha) * tau ** 2 * (logp.exp() * (logp - logq.gather(1, at))).sum(dim=1)
        g = (1 - alpha) * tau * logq.exp()
        g.scatter_add_(1, at, -(1 - alpha) * tau * logp.exp())
        if alpha > 0:
            i = torch.arange(rows.numel(), device=DEV)
            logs = torch.log_softmax(z, dim=1)
            loss[rows] -= alpha * logs[i, s["labels"][rows]]
            g += alpha * logs.exp()
            g[i, s["labels"][rows]] -= alpha
        dz[rows] = g * s["weight"][rows].double()[:, None]
    return loss, dz
