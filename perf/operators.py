"""What the layer's newer operators are timed on: the cases, their plain forms and their values in 64 bits.

Four operators of the sparse MoE layer (8 experts, top-2):

  balance  the router's balance loss and z-loss with per-sequence expert counts, and their gradient to the logits
  train    one training step whose saved pre-activations are 8-bit codes: forward, balance loss, backward
  quant    expert weights [E, K, N] to microscaled 4-bit floating point and back
  mx4      the layer's forward pass on such weights, activations in microscaled 8-bit floating point

`run` computes a plain form in elementary torch operations, or, where `own` is set, calls the library.
"""
import math

import torch

own = False

E, TOP_K = 8, 2
BALANCE_COEF, Z_COEF = 0.01, 0.001


# ------------------------------------------------------------------------------------------------ cases


def listed():
    return [
        # a decode-sized batch: one launch's latency
        {"name": "balance_T32", "op": "balance", "T": 32, "seqs": 1, "mask": False},
        # a packed training batch: ragged sequences, padding tokens masked out
        {"name": "balance_T16384_ragged", "op": "balance", "T": 16384, "seqs": 64, "mask": True},
        # a large global batch, streaming from memory
        {"name": "balance_T1M", "op": "balance", "T": 1 << 20, "seqs": 1000, "mask": True},
        # a step with a few rows per expert
        {"name": "train_T40", "op": "train", "T": 40, "d": 256, "f": 256, "cf": 4.0},
        # the mid layer, with capacity drops
        {"name": "train_mid", "op": "train", "T": 2048, "d": 1536, "f": 8192, "cf": 1.25},
        # the Grok-1 layer, one sequence of 8192 tokens, no drops
        {"name": "train_grok", "op": "train", "T": 8192, "d": 6144, "f": 32768, "cf": 4.0},
        # the mid layer's gate weights, and the Grok-1 layer's down weights
        {"name": "quant_mid", "op": "quant", "K": 1536, "N": 8192},
        {"name": "quant_grok", "op": "quant", "K": 32768, "N": 6144},
        # one token through the mid layer: latency
        {"name": "mx4_T1", "op": "mx4", "T": 1, "d": 1536, "f": 8192, "cf": 4.0},
        # Grok-1 decode: streaming all experts' weights for 32 tokens
        {"name": "mx4_decode", "op": "mx4", "T": 32, "d": 6144, "f": 32768, "cf": 4.0},
        # mid prefill with capacity drops
        {"name": "mx4_mid", "op": "mx4", "T": 2048, "d": 1536, "f": 8192, "cf": 1.25},
        # Grok-1 prefill: bound by the tensor cores
        {"name": "mx4_prefill", "op": "mx4", "T": 8192, "d": 6144, "f": 32768, "cf": 4.0},
    ]


def _spread(rng, lo, hi, step=1):
    """A multiple of step in [lo, hi], spread over its logarithm."""
    v = math.exp(rng.uniform(math.log(lo), math.log(hi + step - 1)))
    return max(lo, min(hi, int(v) // step * step))


def draw(rng):
    op = rng.choice(["balance", "balance", "train", "train", "quant", "mx4", "mx4", "mx4"])
    if op == "balance":
        T = _spread(rng, 1, 1 << 20)
        return {"op": op, "T": T, "seqs": _spread(rng, 1, min(T, 4096)), "mask": rng.random() < 0.7}
    if op == "quant":
        return {"op": op, "K": _spread(rng, 128, 32768, 128), "N": _spread(rng, 128, 6144, 128)}
    return {"op": op, "T": _spread(rng, 1, 8192), "d": _spread(rng, 256, 6144, 256), "f": _spread(rng, 256, 32768, 256),
            "cf": rng.choice([1.0, 1.25, 2.0, 4.0])}


def _capacity(T, cf):
    return min(T, math.ceil(cf * (T * TOP_K) / E))


def work(case):
    op = case["op"]
    if op == "balance":
        T, S = case["T"], case["seqs"]
        # logits and their gradient in fp32, two int32 choices and a mask byte a token, counts a sequence
        return {"bytes": T * (2 * E * 4 + TOP_K * 4 + (1 if case["mask"] else 0)) + S * (E + 1) * 4, "flops": 60.0 * T * E}
    if op == "quant":
        n = E * case["K"] * case["N"]
        return {"bytes": n * (2 + 2), "flops": 4.0 * n}
    T, d, f = case["T"], case["d"], case["f"]
    rows = min(TOP_K * T, E * _capacity(T, case["cf"]))
    used = min(E, TOP_K * T)
    io = 2 * T * d * 2 + E * d * 2
    if op == "mx4":
        return {"bytes": 3 * used * d * f * (0.5 + 1 / 32) + io, "flops": 2.0 * rows * 3 * d * f}
    return {"bytes": 3 * d * f * (used + E) * 2 + 2 * io, "flops": 3 * 2.0 * rows * 3 * d * f}


# ----------------------------------------------------------------------------------------------- inputs


def _generator(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _normal(g, shape, std=1.0):
    return torch.empty(shape, dtype=torch.bfloat16, device="cuda").normal_(0.0, std, generator=g)


def _mx4_codes(w):
    """Codes [E, N, K/2] and scales (in blocks of 128 channels by 128 rows of K) of w [E, K, N]."""
    n_e, K, N = w.shape
    codes = torch.empty((n_e, N, K // 2), dtype=torch.uint8, device="cuda")
    scales = torch.empty((n_e, N // 128, K // 128, 512), dtype=torch.uint8, device="cuda")
    for e in range(n_e):
        v = w[e].t().float().reshape(N, K // 32, 32)
        ex = _shared_exponent(v.abs().amax(-1), 2, 125)
        v = v * _pow2(-ex)[..., None]
        a = v.abs()
        step = torch.where(a < 2, 0.5, torch.where(a < 4, 1.0, 2.0))
        a = (torch.round(a / step) * step).clamp_(max=6.0)
        mag = torch.where(a < 2, a * 2, torch.where(a < 4, a + 2, a / 2 + 4))
        code = (mag + 8 * torch.signbit(v)).to(torch.uint8).reshape(N, K // 2, 2)
        codes[e] = code[..., 0] | code[..., 1] << 4
        s = (ex + 127).to(torch.uint8).reshape(N // 128, 4, 32, K // 128, 4)
        scales[e] = s.permute(0, 3, 2, 1, 4).reshape(N // 128, K // 128, 512)
    return codes, scales


def prepare(case, seed):
    g = _generator(seed)
    op = case["op"]
    if op == "balance":
        T, S = case["T"], case["seqs"]
        logits = torch.empty((T, E), device="cuda").normal_(0.0, 1.5, generator=g)
        idx = logits.topk(TOP_K, dim=1).indices.to(torch.int32)
        # ragged lengths; the tail behind the last sequence is padding
        end = max(1, T - T // 50) if S > 1 else T
        cuts = torch.randint(0, end + 1, (S - 1,), device="cuda", generator=g).sort().values
        offsets = torch.cat([cuts.new_zeros(1), cuts, cuts.new_full((1,), end)]).to(torch.int32)
        mask = torch.rand(T, device="cuda", generator=g) < 0.9 if case["mask"] else None
        return {"op": op, "T": T, "logits": logits, "idx": idx, "offsets": offsets, "mask": mask}
    if op == "quant":
        return {"op": op, "w": _normal(g, (E, case["K"], case["N"]), 1.0 / math.sqrt(case["K"]))}
    T, d, f = case["T"], case["d"], case["f"]
    s = {"op": op, "T": T, "d": d, "f": f, "cf": case["cf"]}
    s["x"] = _normal(g, (T, d))
    s["wr"] = _normal(g, (E, d), 0.02 * math.sqrt(6144 / d))
    # tokens whose second and third logits are within 1e-3 take the row of one that is not: the choice of
    # experts then does not hang on the order in which a logit is summed
    logits = (s["x"].double() @ s["wr"].double().t()).sort(dim=1, descending=True).values
    gap = logits[:, 1] - logits[:, 2]
    s["x"] = torch.where((gap < 1e-3)[:, None], s["x"][gap.argmax()], s["x"])
    shapes = {"wg": (E, d, f), "wu": (E, d, f), "wd": (E, f, d)}
    for k, shape in shapes.items():
        w = _normal(g, shape, 1.0 / math.sqrt(shape[1]))
        s[k] = _mx4_codes(w) if op == "mx4" else w
    if op == "train":
        s["dout"] = _normal(g, (T, d))
        s["offsets"] = torch.tensor([0, T], dtype=torch.int32, device="cuda")
    return s


# --------------------------------------------------------------------------------------- the plain forms


def _pow2(ex):
    """2 ** ex in fp32, exactly, for whole ex in [-127, 127]."""
    return ((ex.clamp(min=-126).int() + 127) << 23).view(torch.float32) * torch.where(ex < -126, 0.5, 1.0)


def _shared_exponent(amax, emax, top):
    """Exponent of a block's shared scale: floor(log2 amax) - emax, one more where amax is over 1.75 powers of
    two (it would round past the largest code), within [-127, top]."""
    m, ex = torch.frexp(amax)
    ex = ex - 1 - emax + (m > 0.875).to(ex.dtype)
    return torch.where(amax > 0, ex, torch.full_like(ex, -127)).clamp(-127, top)


def _mx4_weight(codes, scales):
    """One expert's weights [N, K] in fp32 from its codes [N, K/2] and scales."""
    N, K = codes.shape[0], 2 * codes.shape[1]
    c = torch.stack([codes & 15, codes >> 4], -1).reshape(N, K)
    a = (c & 7).float()
    a = torch.where(a < 4, a * 0.5, torch.where(a < 6, a - 2, 2 * a - 8))
    v = torch.where(c >= 8, -a, a).reshape(N, K // 32, 32)
    ex = scales.reshape(N // 128, K // 128, 32, 4, 4).permute(0, 3, 2, 1, 4).reshape(N, K // 32).int() - 127
    return (v * _pow2(ex)[..., None]).reshape(N, K)


def _mx8(v):
    """v in microscaled 8-bit floating point (e4m3, one power-of-two scale for 32 values), as the values it stands for."""
    b = v.reshape(v.shape[0], -1, 32)
    ex = _shared_exponent(b.abs().amax(-1), 8, 127)[..., None]
    return ((b * _pow2(-ex)).to(torch.float8_e4m3fn).float() * _pow2(ex)).reshape(v.shape)


def _int8(v):
    """v in 8-bit codes (one bf16 scale for 32 values), as the values they stand for."""
    b = v.reshape(v.shape[0], -1, 32)
    s = (b.abs().amax(-1, keepdim=True) / 127).to(torch.bfloat16).float()
    c = torch.round(b / s).clamp(-127, 127)
    return torch.where(s > 0, c * s, torch.zeros_like(b)).reshape(v.shape)


def _balance(logits, idx, offsets, mask):
    T, S = logits.shape[0], offsets.numel() - 1
    t = torch.arange(T, device="cuda")
    seq = torch.searchsorted(offsets[1:].long(), t, right=True)
    live = (t >= offsets[0]) & (seq < S)
    if mask is not None:
        live = live & mask
    seq = torch.where(live, seq, torch.full_like(seq, S))  # row S collects what does not count
    top = logits.amax(1, keepdim=True)
    z = (logits - top).exp()
    total = z.sum(1, keepdim=True)
    p, lse = z / total, (total.log() + top)[:, 0]
    hot = (idx.long()[:, :, None] == torch.arange(E, device="cuda")).sum(1)
    counts = torch.zeros((S + 1, E), dtype=torch.int64, device="cuda").index_add_(0, seq, hot)
    share = counts.double() / counts.sum(1, keepdim=True).clamp(min=1)
    n = live.sum().clamp(min=1)
    ft = share[seq].float()
    dot = (ft * p).sum(1)
    lv = live.double()
    balance = E * (dot.double() * lv).sum() / n
    zloss = (lse.double().square() * lv).sum() / n
    loss = torch.stack([BALANCE_COEF * balance + Z_COEF * zloss, balance, zloss]).float()
    dlogits = p * (BALANCE_COEF * E / n * (ft - dot[:, None]) + 2 * Z_COEF / n * lse[:, None])
    return loss, counts[:S].to(torch.int32), torch.where(live[:, None], dlogits, torch.zeros_like(dlogits)).float()


def _route(x, wr, cf):
    """Logits, the two choices and their weights, and which of them fit the experts' capacity."""
    logits = x @ wr.t()
    first = logits.argmax(1)
    second = logits.scatter(1, first[:, None], -math.inf).argmax(1)
    idx = torch.stack([first, second], 1)
    l2 = logits.gather(1, idx)
    w = (l2 - l2[:, :1]).exp()
    w = w / w.sum(1, keepdim=True)
    hot = (idx[:, :, None] == torch.arange(E, device="cuda")).long()
    before = hot.sum(1).cumsum(0) - hot.sum(1)
    kept = before.gather(1, idx) < _capacity(x.shape[0], cf)
    return logits, idx, w, kept


def _silu(v):
    return v / (1 + (-v).exp())


def _plain_mx4(s):
    x = s["x"].float()
    _, idx, w, kept = _route(x, s["wr"].float(), s["cf"])
    out = torch.zeros_like(x)
    for e in range(E):
        t, j = ((idx == e) & kept).nonzero(as_tuple=True)
        if t.numel() == 0:
            continue
        a = _mx8(x[t])
        h = _silu(a @ _mx4_weight(s["wg"][0][e], s["wg"][1][e]).t()) * (a @ _mx4_weight(s["wu"][0][e], s["wu"][1][e]).t())
        out.index_add_(0, t, w[t, j][:, None] * (_mx8(h) @ _mx4_weight(s["wd"][0][e], s["wd"][1][e]).t()))
    return {"out": out.to(torch.bfloat16)}


def _plain_train(s):
    x, wr, dout = s["x"].float(), s["wr"].float(), s["dout"].float()
    logits, idx, w, kept = _route(x, wr, s["cf"])
    loss, counts, dlogits = _balance(logits, idx, s["offsets"], None)
    out, dx, dw = torch.zeros_like(x), torch.zeros_like(x), torch.zeros_like(w)
    grads = {k: torch.zeros_like(s[k]) for k in ("wg", "wu", "wd")}
    for e in range(E):
        t, j = ((idx == e) & kept).nonzero(as_tuple=True)
        if t.numel() == 0:
            continue
        wg, wu, wd = s["wg"][e].float(), s["wu"][e].float(), s["wd"][e].float()
        a, r, do = x[t], w[t, j][:, None], dout[t]
        g, u = a @ wg, a @ wu
        out.index_add_(0, t, r * ((_silu(g) * u) @ wd))
        g, u = _int8(g), _int8(u)  # what the checkpoint holds
        sg = 1 / (1 + (-g).exp())
        h, dh = g * sg * u, do @ wd.t()
        dw[t, j] = (dh * h).sum(1)
        grads["wd"][e] = (h.t() @ (r * do)).to(torch.bfloat16)
        dh = r * dh
        dg, du = dh * u * sg * (1 + g * (1 - sg)), dh * g * sg
        grads["wg"][e] = (a.t() @ dg).to(torch.bfloat16)
        grads["wu"][e] = (a.t() @ du).to(torch.bfloat16)
        dx.index_add_(0, t, dg @ wg.t() + du @ wu.t())
    dlogits.scatter_add_(1, idx, w * (dw - (w * dw).sum(1, keepdim=True)))
    dx += dlogits @ wr
    half = torch.bfloat16
    return {"out": out.to(half), "loss": loss, "counts": counts, "dx": dx.to(half), "dw_router": (dlogits.t() @ x).to(half),
            "dbias": dlogits.sum(0).to(half), "dw_gate": grads["wg"], "dw_up": grads["wu"], "dw_down": grads["wd"]}


def _plain_quant(s):
    out = torch.empty_like(s["w"])
    for e in range(E):
        b = s["w"][e].float().reshape(-1, 32, s["w"].shape[2])
        ex = _shared_exponent(b.abs().amax(1), 2, 125)[:, None]
        v = b * _pow2(-ex)
        a = v.abs()
        step = torch.where(a < 2, 0.5, torch.where(a < 4, 1.0, 2.0))
        a = (torch.round(a / step) * step).clamp(max=6.0)
        out[e] = (torch.where(v < 0, -a, a) * _pow2(ex)).reshape(out[e].shape).to(torch.bfloat16)
    return {"w": out}


# -------------------------------------------------------------------------------------------------- run


def _run_own(s):
    import sparse_moe_layer_07_b200 as moe

    op = s["op"]
    if op == "balance":
        r = moe.balance_loss(moe.Config(s["T"], 256, 256), s["logits"], s["idx"], token_mask=s["mask"],
                             seq_offsets=s["offsets"], balance_coef=BALANCE_COEF, z_coef=Z_COEF)
        return {"loss": r["loss"], "counts": r["counts"], "dlogits": r["dlogits"]}
    if op == "quant":
        cfg = moe.Config(0, 256, 256)
        return {"w": moe.dequantize_mx4(cfg, *moe.quantize_mx4(cfg, s["w"]))}
    cfg = moe.Config(s["T"], s["d"], s["f"], capacity_factor=s["cf"])
    if op == "mx4":
        qw = moe.MxExperts.from_codes(*s["wg"], *s["wu"], *s["wd"])
        return {"out": moe.layer_forward_mx4(cfg, s["x"], s["wr"], qw)}
    weights = (s["wr"], s["wg"], s["wu"], s["wd"])
    ckpt = torch.empty(moe.checkpoint_size_c8(cfg), dtype=torch.uint8, device="cuda")
    ws = torch.empty(moe.workspace_size_train_c8(cfg), dtype=torch.uint8, device="cuda")
    out = moe.layer_forward_train_c8(cfg, s["x"], *weights, ckpt, ws)
    kept = moe.checkpoint_views_c8(cfg, ckpt)
    b = moe.balance_loss(cfg, kept["logits"], kept["topk_idx"], seq_offsets=s["offsets"], balance_coef=BALANCE_COEF,
                         z_coef=Z_COEF)
    g = moe.layer_backward_c8(cfg, s["x"], *weights, s["dout"], ckpt, ws, dlogits=b["dlogits"])
    return {"out": out, "loss": b["loss"], "counts": b["counts"], "dx": g["dx"], "dw_router": g["dw_router"],
            "dbias": g["dbias"], "dw_gate": g["dw_gate"], "dw_up": g["dw_up"], "dw_down": g["dw_down"]}


def run(s):
    if own:
        return _run_own(s)
    op = s["op"]
    if op == "balance":
        loss, counts, dlogits = _balance(s["logits"], s["idx"], s["offsets"], s["mask"])
        return {"loss": loss, "counts": counts, "dlogits": dlogits}
    return _plain_quant(s) if op == "quant" else _plain_mx4(s) if op == "mx4" else _plain_train(s)


# ------------------------------------------------------------------------------------ values in 64 bits


def _exact_balance(logits, idx, offsets, mask):
    logits = logits.double()
    T, S = logits.shape[0], offsets.numel() - 1
    bounds = offsets.long()
    live = torch.zeros(T, dtype=torch.bool, device="cuda")
    live[int(bounds[0]):int(bounds[-1])] = True
    if mask is not None:
        live &= mask
    lens = bounds[1:] - bounds[:-1]
    seq = torch.zeros(T, dtype=torch.int64, device="cuda")
    seq[int(bounds[0]):int(bounds[-1])] = torch.repeat_interleave(torch.arange(S, device="cuda"), lens)
    lse = torch.logsumexp(logits, 1)
    p = torch.exp(logits - lse[:, None])
    keys = (seq[:, None] * E + idx.long())[live].reshape(-1)
    counts = torch.bincount(keys, minlength=S * E).reshape(S, E)
    n = int(live.sum())
    if n == 0:
        return torch.zeros(3, dtype=torch.float64), counts.to(torch.int32), torch.zeros_like(logits)
    per = counts.sum(1, keepdim=True) / TOP_K  # tokens of a sequence
    f = torch.where(per > 0, counts / (TOP_K * per).clamp(min=1), torch.zeros_like(per))
    psum = torch.zeros((S, E), dtype=torch.float64, device="cuda").index_add_(0, seq[live], p[live])
    balance = E * (f * psum).sum() / n
    zloss = (lse[live] ** 2).sum() / n
    jac = p * f[seq] - p * (p * f[seq]).sum(1, keepdim=True)
    grad = BALANCE_COEF * E / n * jac + Z_COEF * 2 / n * lse[:, None] * p
    grad[~live] = 0
    return torch.stack([BALANCE_COEF * balance + Z_COEF * zloss, balance, zloss]), counts.to(torch.int32), grad


_E2M1 = [0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0]


def _two(e):
    """2 ** e in fp64, to the last bit (pow is not)."""
    return ((e.long() + 1023) << 52).view(torch.float64)


def _exact_scale(amax, emax, top):
    e = torch.floor(torch.log2(amax.clamp(min=2.0 ** -200)))
    e = torch.where(amax >= _two(e + 1), e + 1, torch.where(amax < _two(e), e - 1, e))
    return _two((torch.where(amax > 1.75 * _two(e), e + 1, e) - emax).clamp(-127, top))


def _exact_mx8(v):
    b = v.reshape(v.shape[0], -1, 32)
    x = _exact_scale(b.abs().amax(2, keepdim=True), 8, 127)
    b = b / x
    ulp = _two(torch.floor(torch.log2(b.abs().clamp(min=2.0 ** -6))) - 3)
    return (torch.round(b / ulp) * ulp * x).reshape(v.shape)


def _exact_weight(codes, scales):
    table = torch.tensor(_E2M1 + [-v for v in _E2M1], dtype=torch.float64, device="cuda")
    N, K = codes.shape[0], 2 * codes.shape[1]
    w = torch.empty((N, K), dtype=torch.float64, device="cuda")
    w[:, 0::2], w[:, 1::2] = table[(codes % 16).int()], table[(codes // 16).int()]
    n, k = torch.arange(N, device="cuda")[:, None], torch.arange(0, K, 32, device="cuda")[None]
    at = ((n // 128) * (K // 128) + k // 128) * 512 + (n % 32) * 16 + (n % 128) // 32 * 4 + k % 128 // 32
    return w.reshape(N, -1, 32).mul_(_two(scales.reshape(-1)[at].long() - 127)[..., None]).reshape(N, K)


def _exact_slots(s):
    """The router in 64 bits: logits, and for each expert its kept tokens with their weights."""
    x, T = s["x"].double(), s["T"]
    logits = x @ s["wr"].double().t()
    l2, idx = logits.sort(dim=1, descending=True, stable=True)
    idx, w = idx[:, :TOP_K], torch.softmax(l2[:, :TOP_K], 1)
    groups = []
    for e in range(E):
        t, j = (idx == e).nonzero(as_tuple=True)
        m = _capacity(T, s["cf"])
        groups.append((t[:m], j[:m], w[t[:m], j[:m]]))
    return x, logits, idx, w, groups


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "balance":
        loss, counts, grad = _exact_balance(s["logits"], s["idx"], s["offsets"], s["mask"])
        return {"loss": loss, "counts": counts, "dlogits": grad}
    if op == "quant":
        out = torch.empty(s["w"].shape, dtype=torch.float64, device="cuda")
        mids = torch.tensor([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0], dtype=torch.float64, device="cuda")
        table = torch.tensor(_E2M1, dtype=torch.float64, device="cuda")
        for e in range(E):
            b = s["w"][e].double().reshape(-1, 32, out.shape[2])
            x = _exact_scale(b.abs().amax(1, keepdim=True), 2, 125)
            v = (b / x).abs()
            low, high = torch.bucketize(v, mids), torch.bucketize(v, mids, right=True)
            # on a midpoint the two differ, and the even code is the nearer
            code = torch.where(low == high, low, torch.where(low % 2 == 0, low, high))
            out[e] = (torch.sign(b) * table[code] * x).reshape(out[e].shape)
        return {"w": out}
    x, logits, idx, w, groups = _exact_slots(s)
    out = torch.zeros_like(x)
    if op == "mx4":
        for e, (t, _, r) in enumerate(groups):
            if t.numel() == 0:
                continue
            a = _exact_mx8(x[t])
            g = a @ _exact_weight(s["wg"][0][e], s["wg"][1][e]).t()
            u = a @ _exact_weight(s["wu"][0][e], s["wu"][1][e]).t()
            y = _exact_mx8(g * torch.sigmoid(g) * u) @ _exact_weight(s["wd"][0][e], s["wd"][1][e]).t()
            out[t] += r[:, None] * y
        return {"out": out}
    loss, counts, dl = _exact_balance(logits, idx, s["offsets"], None)
    dout, dx = s["dout"].double(), torch.zeros_like(x)
    dwt = torch.zeros_like(w)
    grads = {k: torch.zeros(s[k].shape, dtype=torch.float64, device="cuda") for k in ("wg", "wu", "wd")}
    for e, (t, j, r) in enumerate(groups):
        if t.numel() == 0:
            continue
        wg, wu, wd = s["wg"][e].double(), s["wu"][e].double(), s["wd"][e].double()
        a, do = x[t], dout[t]
        pre = [a @ wg, a @ wu]
        out[t] += r[:, None] * ((pre[0] * torch.sigmoid(pre[0]) * pre[1]) @ wd)
        for i in range(2):  # 8-bit codes in blocks of 32 with a bf16 scale
            b = pre[i].unflatten(1, (-1, 32))
            q = (b.abs().max(2, keepdim=True).values / 127).to(torch.bfloat16).double()
            pre[i] = torch.nan_to_num(torch.clip(torch.round(b / q), -127, 127) * q).flatten(1)
        g, u = pre
        sig = torch.sigmoid(g)
        back = do @ wd.t()
        act = g * sig
        dwt[t, j] = torch.einsum("rf,rf,rf->r", back, act, u)
        grads["wd"][e] = (act * u * r[:, None]).t() @ do
        back *= r[:, None]
        dg, du = back * u * (sig + act * (1 - sig)), back * act
        grads["wg"][e], grads["wu"][e] = a.t() @ dg, a.t() @ du
        dx[t] += dg @ wg.t() + du @ wu.t()
    soft = torch.diag_embed(w) - w[:, :, None] * w[:, None, :]
    for j in range(TOP_K):
        dl[torch.arange(s["T"], device="cuda"), idx[:, j]] += (soft[:, j] * dwt).sum(1)
    return {"out": out, "loss": loss, "counts": counts, "dx": dx + dl @ s["wr"].double(), "dw_router": dl.t() @ x,
            "dbias": dl.sum(0), "dw_gate": grads["wg"], "dw_up": grads["wu"], "dw_down": grads["wd"]}
