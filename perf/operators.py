"""Timed cases of five operators around the QLoRA linear layer, each with a
plain torch form and an exact form in 64 bits:

  act8          8-bit activation checkpoints: store a bf16 activation as E4M3
                codes with one power-of-two scale per 32 values, and restore it
  swiglu        the gated activation between gate/up and down, its backward
                taking gate and up from 8-bit checkpoints
  bwd_act8      backward of the LoRA linear layer from an 8-bit checkpoint of X
  q4g_quantize  4-bit weights with group scales: quantize and expand
  q4g_linear    Y = X W'^T on such a weight, one to 64 tokens

``own`` False computes the plain form, True calls the library.
"""

import torch

own = False

DEV = "cuda"

# the sixteen NF4 values, ascending
NF4 = (-1.0, -0.6961928009986877, -0.5250730514526367, -0.39491748809814453, -0.28444138169288635,
       -0.18477343022823334, -0.09105003625154495, 0.0, 0.07958029955625534, 0.16093020141124725,
       0.24611230194568634, 0.33791524171829224, 0.44070982933044434, 0.5626170039176941, 0.7229568362236023, 1.0)


# ---------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------
def listed():
    return [
        # the input of a 7B attention block for one 1024-token sequence
        {"name": "act8 1024x4096", "op": "act8", "T": 1024, "K": 4096},
        # the input of a 7B down projection, a batch of 4096 tokens
        {"name": "act8 4096x11008", "op": "act8", "T": 4096, "K": 11008},
        # a short prompt through the 7B MLP (odd token count)
        {"name": "swiglu 77x11008", "op": "swiglu", "T": 77, "F": 11008},
        # the 65B-shaped MLP at a training batch
        {"name": "swiglu 4096x22016", "op": "swiglu", "T": 4096, "F": 22016},
        # first layer of the stack: adapter gradients only, no input gradient
        {"name": "bwd attn T1024 r16 no dX", "op": "bwd_act8", "T": 1024, "N": 4096, "K": 4096, "r": 16,
         "dx": False, "p": 0.0},
        # 7B gate projection with adapter dropout
        {"name": "bwd gate T1000 r16 p.05", "op": "bwd_act8", "T": 1000, "N": 11008, "K": 4096, "r": 16,
         "dx": True, "p": 0.05},
        # 7B down projection at a training batch, rank 64
        {"name": "bwd down T4096 r64", "op": "bwd_act8", "T": 4096, "N": 4096, "K": 11008, "r": 64,
         "dx": True, "p": 0.0},
        # a merged bf16 7B MLP weight brought to 4 bits for serving
        {"name": "q4g quant 11008x4096 g128", "op": "q4g_quantize", "N": 11008, "K": 4096, "group": 128,
         "sym": False, "f32": False},
        # an fp32 attention weight, fine symmetric groups
        {"name": "q4g quant 4096x4096 g32 f32", "op": "q4g_quantize", "N": 4096, "K": 4096, "group": 32,
         "sym": True, "f32": True},
        # decode of one token, 7B attention projection: latency
        {"name": "q4g 4096x4096 T1 g128", "op": "q4g_linear", "T": 1, "N": 4096, "K": 4096, "group": 128,
         "sym": False},
        # decode of one token, 65B-shaped up projection: bandwidth
        {"name": "q4g 22016x8192 T1 g128", "op": "q4g_linear", "T": 1, "N": 22016, "K": 8192, "group": 128,
         "sym": False},
        # a decode batch of 37 sequences, 7B gate, fine symmetric groups
        {"name": "q4g 11008x4096 T37 g32", "op": "q4g_linear", "T": 37, "N": 11008, "K": 4096, "group": 32,
         "sym": True},
    ]


def _log(rng, lo, hi):
    """An integer in [lo, hi], its logarithm uniform."""
    return min(hi, max(lo, int(round(lo * (hi / lo) ** rng.random()))))


def draw(rng):
    op = rng.choice(["act8", "swiglu", "bwd_act8", "q4g_quantize", "q4g_linear"])
    if op == "act8":
        return {"op": op, "T": _log(rng, 1, 4096), "K": 32 * _log(rng, 2, 344)}
    if op == "swiglu":
        return {"op": op, "T": _log(rng, 1, 4096), "F": 32 * _log(rng, 2, 688)}
    if op == "bwd_act8":
        return {"op": op, "T": _log(rng, 1, 2048), "N": 8 * _log(rng, 8, 1376), "K": 64 * _log(rng, 1, 128),
                "r": rng.choice([3, 8, 16, 33, 64, 128]), "dx": rng.random() < 0.5,
                "p": rng.choice([0.0, 0.0, 0.05, 0.1])}
    group = rng.choice([32, 64, 128])
    if op == "q4g_quantize":
        return {"op": op, "N": _log(rng, 1, 8192), "K": 8 * _log(rng, 4, 1376), "group": group,
                "sym": rng.random() < 0.5, "f32": rng.random() < 0.5}
    return {"op": op, "T": _log(rng, 1, 64), "N": _log(rng, 7, 11008), "K": 8 * _log(rng, 4, 1376), "group": group,
            "sym": rng.random() < 0.5}


def work(case):
    op = case["op"]
    if op == "act8":  # store: 2 B in, 1 + 1/32 out; restore: the reverse
        n = case["T"] * case["K"]
        return {"bytes": n * (4 + 2 * 33 / 32), "flops": 2 * n}
    if op == "swiglu":
        # forward: two bf16 in, one out, two checkpoints out; backward: two checkpoints and dH in, two bf16 out
        n = case["T"] * case["F"]
        return {"bytes": n * (6 + 2 * 33 / 32) + n * (6 + 2 * 33 / 32), "flops": 16 * n}
    if op == "bwd_act8":
        T, N, K, r = case["T"], case["N"], case["K"], case["r"]
        b = T * K * 33 / 32 + 2 * T * N + 4 * T * r + 2 * r * N + 4 * r * (N + K)
        f = 4 * T * N * r + 2 * T * K * r
        if case["dx"]:
            b += N * K * (0.5 + 1 / 64) + 2 * T * K + 2 * r * K
            f += 2 * T * N * K + 2 * T * K * r
        if case["p"] > 0:
            b += T * K / 8
        return {"bytes": b, "flops": f}
    N, K = case["N"], case["K"]
    groups = N * -(-K // case["group"])
    coded = N * K / 2 + groups * (2 if case["sym"] else 3)
    if op == "q4g_quantize":
        return {"bytes": N * K * (4 if case["f32"] else 2) + 2 * coded + 2 * N * K, "flops": 4 * N * K}
    return {"bytes": coded + 2 * case["T"] * (N + K), "flops": 2 * case["T"] * N * K}


# ---------------------------------------------------------------------------
# plain forms
# ---------------------------------------------------------------------------
def _pow2(k):
    """2^k as fp32 for int32 k in the normal range."""
    return ((k + 127) << 23).view(torch.float32)


def _act8_store(x):
    """Codes (float8_e4m3fn [T, K]) and exponents k (int32 [T, K/32])."""
    T, K = x.shape
    v = x.float().view(T, K // 32, 32)
    a = torch.where(torch.isfinite(v), v.abs(), torch.zeros_like(v)).amax(dim=2)
    bits = a.view(torch.int32)
    k = ((bits >> 23) - 135 + ((bits & 0x7FFFFF) > 0x600000).int()).clamp(min=-124)
    codes = (v / _pow2(k)[:, :, None]).to(torch.float8_e4m3fn)
    return codes.view(T, K), k


def _act8_load(codes, k):
    """fp32 [T, K]."""
    T, K = codes.shape
    return (codes.float().view(T, K // 32, 32) * _pow2(k)[:, :, None]).view(T, K)


def _nf4_expand(s):
    """W' as fp32 values, rounded to bf16 once (the weight the layer multiplies with)."""
    p = s["packed"]
    c = torch.stack([p >> 4, p & 15], dim=1).view(-1, 64).long()
    e = s["c8"].view(torch.float8_e4m3fn).float().view(-1)
    groups = s["dq_scale"].repeat_interleave(256)[: e.numel()]
    a = e * groups + s["dq_mean"]
    w = torch.tensor(NF4, device=DEV)[c] * a[:, None]
    return w.to(torch.bfloat16).float().view(s["N"], s["K"])


def _keep_bits(packed, K):
    bits = torch.arange(8, device=packed.device, dtype=torch.int32)
    return ((packed.int()[:, :, None] >> bits) & 1).view(packed.shape[0], K)


def _sigmoid(g):
    return 1.0 / (1.0 + torch.exp(-g))


def _pad_groups(w, group):
    N, K = w.shape
    g = -(-K // group)
    return torch.nn.functional.pad(w, (0, g * group - K)).view(N, g, group)


def _divide(a, b):
    """fp32 quotient, correctly rounded (through fp64)."""
    return (a.double() / b.double()).float()


def _q4g_store(W, group, sym):
    """Codes [N, groups, group] (int32), bf16 scale and uint8 zero [N, groups].
    The zeros that pad a short last group do not move its range (it holds 0)."""
    w = _pad_groups(W.float(), group)
    if sym:
        s = _divide(w.abs().amax(dim=2), torch.full((), 7.0, device=w.device))
    else:
        lo, hi = w.amin(dim=2).clamp(max=0), w.amax(dim=2).clamp(min=0)
        s = _divide(hi - lo, torch.full((), 15.0, device=w.device))
    s = s.to(torch.bfloat16)
    s = torch.where(s.float() < 2.0 ** -126, torch.zeros_like(s), s)
    live = s > 0
    d = torch.where(live, s.float(), torch.ones_like(s, dtype=torch.float32))
    z = torch.full_like(d, 8.0) if sym else torch.where(live, torch.round(_divide(-lo, d)).clamp(0, 15),
                                                       torch.full_like(d, 8.0))
    q = (torch.round(_divide(w, d[:, :, None])) + z[:, :, None]).clamp(0, 15)
    q = torch.where(live[:, :, None], q, torch.full_like(q, 8.0))
    return q.int(), s, z.to(torch.uint8)


def _q4g_load(q, s, z, K):
    """W' fp32 [N, K] = s (q - z)."""
    w = (q.float() - z.float()[:, :, None]) * s.float()[:, :, None]
    return w.view(q.shape[0], -1)[:, :K]


def _q4g_pack(q, K):
    """uint8 [N, 16 ceil(K/32)]: element e of a row in byte e/2, even e in the high nibble."""
    N = q.shape[0]
    q = q.view(N, -1)[:, :K]
    q = torch.nn.functional.pad(q, (0, -K % 32)).view(N, -1, 2)
    return (q[:, :, 0] * 16 + q[:, :, 1]).to(torch.uint8)


def _q4g_unpack(packed, K, group):
    q = torch.stack([packed >> 4, packed & 15], dim=2).view(packed.shape[0], -1)[:, :K].int()
    return _pad_groups(q, group)


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------
def _randn(gen, *shape):
    return torch.randn(*shape, generator=gen, device=DEV)


def _activation(gen, T, K):
    """bf16 activations with a few large channels, as transformer layers have."""
    x = _randn(gen, T, K)
    big = torch.rand(K, generator=gen, device=DEV) < 0.005
    return torch.where(big, 20 * x, x).to(torch.bfloat16)


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


def prepare(case, seed):
    gen = torch.Generator(device=DEV)
    gen.manual_seed(int(seed))
    s = dict(case)
    op = case["op"]
    if op == "act8":
        s["X"] = _activation(gen, case["T"], case["K"])
    elif op == "swiglu":
        s["gate"] = (2 * _randn(gen, case["T"], case["F"])).to(torch.bfloat16)
        s["up"] = _randn(gen, case["T"], case["F"]).to(torch.bfloat16)
        s["dH"] = _randn(gen, case["T"], case["F"]).to(torch.bfloat16)
    elif op == "bwd_act8":
        T, N, K, r = case["T"], case["N"], case["K"], case["r"]
        s.update(_nf4_weight(gen, N, K))
        x = _activation(gen, T, K)
        s["dY"] = _randn(gen, T, N).to(torch.bfloat16)
        s["A"] = (_randn(gen, r, K) / 64).to(torch.bfloat16)
        s["B"] = (0.01 * _randn(gen, N, r)).to(torch.bfloat16)
        s["scale"] = 16.0 / r
        codes, k = _act8_store(x)  # what the forward left: the checkpoint of X and U
        s["codes"], s["xscale"] = codes.view(torch.uint8), (k + 127).to(torch.uint8)
        if case["p"] > 0:
            on = (torch.rand(T, K, generator=gen, device=DEV) >= case["p"]).int()
            bits = torch.arange(8, device=DEV, dtype=torch.int32)
            s["keep"] = (on.view(T, K // 8, 8) << bits).sum(dim=2).to(torch.uint8)
            s["U"] = ((x.float() * on) @ s["A"].float().T) / (1 - case["p"])
        else:
            s["keep"] = None
            s["U"] = x.float() @ s["A"].float().T
    else:
        W = 0.02 * _randn(gen, case["N"], case["K"])
        if op == "q4g_quantize":
            s["W"] = W if case["f32"] else W.to(torch.bfloat16)
        else:
            q, s["wscale"], zero = _q4g_store(W.to(torch.bfloat16), case["group"], case["sym"])
            s["packed"] = _q4g_pack(q, case["K"])
            s["zero"] = None if case["sym"] else zero
            s["X"] = _activation(gen, case["T"], case["K"])
    if own:  # the handles around these tensors that a program keeps with them
        import bit_nf4_quantized_16_amd as qn
        if op == "bwd_act8":
            s["w"] = qn.NF4Weight(case["N"], case["K"], s["packed"], c8=s["c8"], dq_scale=s["dq_scale"],
                                  dq_mean=s["dq_mean"])
            s["X8"] = qn.Act8(case["T"], case["K"], s["codes"], s["xscale"])
        elif op == "q4g_linear":
            s["w"] = qn.Q4GWeight(case["N"], case["K"], case["group"], s["packed"], s["wscale"], s["zero"])
    return s


# ---------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------
def run(s):
    return _run_own(s) if own else _run_plain(s)


def _run_plain(s):
    op = s["op"]
    if op == "act8":
        return _act8_load(*_act8_store(s["X"])).to(torch.bfloat16)
    if op == "swiglu":
        g, u = s["gate"].float(), s["up"].float()
        h = (g * _sigmoid(g) * u).to(torch.bfloat16)
        g8, u8 = _act8_load(*_act8_store(s["gate"])), _act8_load(*_act8_store(s["up"]))
        d, sg = s["dH"].float(), _sigmoid(g8)
        return h, (d * u8 * sg * (1 + g8 * (1 - sg))).to(torch.bfloat16), (d * g8 * sg).to(torch.bfloat16)
    if op == "bwd_act8":
        x = _act8_load(s["codes"].view(torch.float8_e4m3fn), s["xscale"].int() - 127)
        d, A, B = s["dY"].float(), s["A"].float(), s["B"].float()
        G = s["scale"] * (d @ B)
        c, keep = 1.0, None
        if s["keep"] is not None:
            c, keep = 1.0 / (1.0 - s["p"]), _keep_bits(s["keep"], s["K"])
            x = x * keep
        dA, dB = c * (G.T @ x), s["scale"] * (d.T @ s["U"])
        if not s["dx"]:
            return {"dA": dA, "dB": dB}
        ga = G @ A if keep is None else c * (G @ A) * keep
        return {"dA": dA, "dB": dB, "dX": (d @ _nf4_expand(s) + ga).to(torch.bfloat16)}
    if op == "q4g_quantize":
        q, scale, zero = _q4g_store(s["W"], s["group"], s["sym"])
        return _q4g_load(q, scale, zero, s["K"]).to(torch.bfloat16), scale, zero
    q = _q4g_unpack(s["packed"], s["K"], s["group"])
    zero = s["zero"] if s["zero"] is not None else torch.full(q.shape[:2], 8, dtype=torch.uint8, device=DEV)
    return (s["X"].float() @ _q4g_load(q, s["wscale"], zero, s["K"]).T).to(torch.bfloat16)


def _run_own(s):
    import bit_nf4_quantized_16_amd as qn

    op = s["op"]
    if op == "act8":
        return qn.act8_dequantize(qn.act8_quantize(s["X"]))
    if op == "swiglu":
        h, g8, u8, _ = qn.swiglu_fwd(s["gate"], s["up"])
        dg, du = qn.swiglu_bwd(g8, u8, s["dH"])
        return h, dg, du
    if op == "bwd_act8":
        dX, dA, dB = qn.qlora_linear_bwd_act8(s["w"], s["X8"], s["dY"], s["A"], s["B"], s["scale"], U=s["U"],
                                              need_dx=s["dx"], keep=s["keep"], p=s["p"])
        return {"dA": dA, "dB": dB, "dX": dX} if s["dx"] else {"dA": dA, "dB": dB}
    if op == "q4g_quantize":
        w = qn.q4g_quantize(s["W"], group=s["group"], symmetric=s["sym"])
        zero = w.zero if w.zero is not None else torch.full(w.scale.shape, 8, dtype=torch.uint8, device=DEV)
        return qn.q4g_dequantize(w), w.scale, zero
    return qn.q4g_linear_fwd(s["w"], s["X"])


# ---------------------------------------------------------------------------
# the definitions in 64 bits
# ---------------------------------------------------------------------------
def _p2(k):
    """2^k in fp64 for integer k."""
    return ((k.long() + 1023) << 52).view(torch.float64)


def _exact_act8(x):
    """Every finite value on its block's E4M3 grid, from the real-number
    definition: 3 fraction bits, smallest step 2^-9, all times 2^k."""
    v = x.double().view(x.shape[0], -1, 32)
    a = v.abs().amax(dim=2, keepdim=True)
    m, e = torch.frexp(a)  # a = m 2^e, m in [1/2, 1)
    k = torch.where(a > 0, e - 9 + (m > 0.875).int(), torch.full_like(e, -124)).clamp(min=-124)
    y = v * _p2(-k)
    step = _p2((torch.frexp(y)[1] - 1).clamp(min=-6) - 3)
    return (torch.round(y / step) * step * _p2(k)).view(x.shape)


def _exact_e4m3(c):
    """E4M3 codes (uint8) as fp64 values."""
    c = c.int()
    e, m = (c >> 3) & 15, (c & 7).double()
    v = torch.where(e == 0, m * 2.0 ** -9, (1 + m / 8) * _p2(e - 7))
    return torch.where(c >= 128, -v, v)


def _exact_x8(s):
    v = _exact_e4m3(s["codes"]).view(s["T"], -1, 32)
    return (v * _p2(s["xscale"].int()[:, :, None] - 127)).view(s["T"], s["K"])


def _exact_nf4(s):
    """W' [N, K]: the stored codes and constants, rounded as the weight's
    definition says (a' = fl32(fl32(E S) + mean), w' = bf16(fl32(T a')))."""
    hi, lo = s["packed"] >> 4, s["packed"] & 15
    c = torch.stack([hi, lo], dim=1).view(-1).long()
    e = _exact_e4m3(s["c8"])
    idx = torch.arange(e.numel(), device=DEV) // 256
    a = ((e * s["dq_scale"].double()[idx]).float().double() + s["dq_mean"].double()).float().double()
    w = (torch.tensor(NF4, device=DEV, dtype=torch.float32).double()[c].view(-1, 64) * a[:, None]).float()
    return w.to(torch.bfloat16).double().view(s["N"], s["K"])


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "act8":
        return _exact_act8(s["X"])
    if op == "swiglu":
        g, u, d = s["gate"].double(), s["up"].double(), s["dH"].double()
        g8, u8 = _exact_act8(s["gate"]), _exact_act8(s["up"])
        p = torch.sigmoid(g8)
        return g * torch.sigmoid(g) * u, d * u8 * (p + g8 * p * (1 - p)), d * g8 * p
    if op == "bwd_act8":
        d, A, B, U = s["dY"].double(), s["A"].double(), s["B"].double(), s["U"].double()
        G = s["scale"] * torch.mm(d, B)
        x = _exact_x8(s)
        mask = 1.0
        if s["keep"] is not None:
            j = torch.arange(s["K"], device=DEV)
            mask = ((s["keep"][:, j // 8].int() >> (j % 8).int()) & 1).double() / (1 - s["p"])
            x = x * mask
        out = {"dA": torch.mm(G.T, x), "dB": s["scale"] * torch.mm(d.T, U)}
        if case["dx"]:
            out["dX"] = torch.mm(d, _exact_nf4(s)) + torch.mm(G, A) * mask
        return out
    N, K, group = case["N"], case["K"], case["group"]
    at = torch.arange(K, device=DEV) // group
    if op == "q4g_quantize":
        W = s["W"].double()
        n = int(at[-1]) + 1
        idx = at.expand(N, K)
        zeros = torch.zeros(N, n, dtype=torch.float64, device=DEV)
        hi = zeros.scatter_reduce(1, idx, W, "amax", include_self=True)
        lo = zeros.scatter_reduce(1, idx, W, "amin", include_self=True)
        step = (torch.maximum(hi, -lo) / 7 if case["sym"] else (hi - lo) / 15).float().to(torch.bfloat16).double()
        d = torch.where(step > 0, step, torch.ones_like(step))
        z = torch.full_like(step, 8.0) if case["sym"] else torch.where(step > 0, torch.round(-lo / d), 8.0).clamp(0, 15)
        q = (torch.round(W / d[:, at]) + z[:, at]).clamp(0, 15)
        return step[:, at] * (q - z[:, at]), step, z.to(torch.uint8)
    j = torch.arange(K, device=DEV)
    q = torch.where(j % 2 == 0, s["packed"][:, j // 2] >> 4, s["packed"][:, j // 2] & 15).double()
    z = s["zero"].double()[:, at] if s["zero"] is not None else 8.0
    return torch.mm(s["X"].double(), (s["wscale"].double()[:, at] * (q - z)).T)
