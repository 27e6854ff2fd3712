"""The FP8 and router-training operators as cases that can be timed and checked.

Every case is one call, or one run of calls, that a user of an expert layer makes: the FP8
(E4M3, one scale per 128) grouped product at serving and prefill sizes, the two-projection
expert network around it, one training step of an expert projection (the quantisers, the
product and both of its gradients), the row quantiser, and the router's balance loss with
its counts and gradient.  With ``own`` false ``run`` takes the plain form, elementary torch
operations in 32 bits; with ``own`` true it calls the library.  ``exact`` is the same
definition in 64 bits, written apart from the plain form.
"""
import math

import torch

own = False

BLK = 128      # elements (or tokens) that share one scale
TOP = 448.0    # largest E4M3 value
FP8 = torch.float8_e4m3fn


def listed():
    return [
        # One token of a 256-expert, top-8 layer on one of eight tensor-parallel GPUs: its eight
        # rows meet eight experts' gate/up weights (the latency of a single token).
        dict(name="product 1 token tp8", op="product", T=1, E=256, k=8, N=512, K=6144, skew=0.0),
        # A decode batch on one of eight expert-parallel GPUs: about 32 rows per expert, every
        # weight read once (gate/up projection).
        dict(name="product decode ep8", op="product", T=128, E=32, k=8, N=4096, K=6144, skew=0.0),
        # A prompt on the same GPU: about 512 rows per expert.
        dict(name="product prefill ep8", op="product", T=2048, E=32, k=8, N=4096, K=6144, skew=0.0),
        # A dense projection: one group, a large square product.
        dict(name="product dense", op="product", T=8192, E=1, k=1, N=8192, K=8192, skew=0.0),
        # A small model's odd sizes under a skewed router: ragged scale blocks on both axes,
        # long, short and empty groups.
        dict(name="product ragged skewed", op="product", T=259, E=24, k=3, N=1552, K=2064, skew=1.0),
        # The expert network of a decode batch: quantise, gate/up with SwiGLU and requantisation,
        # down projection.
        dict(name="experts decode ep8", op="experts", T=128, E=32, k=8, N=2048, K=6144, skew=0.0),
        # The same on the tensor-parallel share at a full decode batch: 256 experts, narrow.
        dict(name="experts decode tp8", op="experts", T=1024, E=256, k=8, N=256, K=6144, skew=0.0),
        # One training step of the gate/up projection of 16 local experts, 512 rows each.
        dict(name="train step", op="train", T=2048, E=16, k=4, N=4096, K=6144, skew=0.0),
        # A training step of a small model under a skewed router, ragged in every size.
        dict(name="train step ragged", op="train", T=517, E=12, k=2, N=784, K=1040, skew=1.0),
        # The tokens of a long prompt quantised before the gate/up projection.
        dict(name="quantize tokens", op="quantize", T=16384, K=6144, bf16=True),
        # The router of a prompt batch in training: one balance term over all tokens.
        dict(name="balance batch", op="balance", T=16384, E=256, k=8, S=1, masked=0.0, routed=False),
        # The same per sequence in a padded batch, with the gradient of the routing weights.
        dict(name="balance sequences", op="balance", T=4099, E=160, k=6, S=37, masked=0.1, routed=True),
    ]


def _log(rng, lo, hi, mult=1):
    v = math.exp(rng.uniform(math.log(lo), math.log(hi)))
    return max(lo, min(hi, int(round(v / mult)) * mult))


def draw(rng):
    op = rng.choice(["product", "product", "product", "experts", "train", "quantize", "balance", "balance"])
    skew = rng.choice([0.0, 0.5, 1.0])
    if op == "balance":
        E = _log(rng, 4, 1024)
        return dict(op=op, T=_log(rng, 1, 16384 * 256 // max(E, 256)), E=E, k=rng.randint(1, min(E, 16)), S=_log(rng, 1, 64),
                    masked=rng.choice([0.0, 0.05, 0.5]), routed=rng.random() < 0.5)
    if op == "quantize":
        K = _log(rng, 16, 8192, 16)
        return dict(op=op, T=_log(rng, 1, 16384 * 6144 // 8192), K=K, bf16=rng.random() < 0.7)
    while True:
        E = _log(rng, 1, 256)
        k = rng.randint(1, min(E, 8))
        T = _log(rng, 1, 4096)
        N = _log(rng, 16, 4096, 16) if op != "experts" else _log(rng, 128, 2048, 128)
        K = _log(rng, 16, 8192, 16)
        weights, flops = E * N * K, 2 * T * k * N * K
        if op == "experts":
            weights, flops = 3 * weights, 3 * flops
        if op == "train":
            weights, flops = 4 * weights, 3 * flops
        if weights <= 8e8 and flops <= 8e11 and E * T * k * max(N, K) <= 3e10:
            return dict(op=op, T=T, E=E, k=k, N=N, K=K, skew=skew)


# ---- inputs ---------------------------------------------------------------------------------

def _generator(seed):
    return torch.Generator(device="cuda").manual_seed(int(seed))


def _encode(x):
    """FP8 codes and scales of x [..., C], one scale per 128 along C (made ready inputs)."""
    C = x.shape[-1]
    n = -(-C // BLK)
    b = torch.nn.functional.pad(x.float(), (0, n * BLK - C)).unflatten(-1, (n, BLK))
    s = b.abs().amax(-1) / TOP
    q = torch.where(s[..., None] > 0, b / s[..., None], 0.0).clamp(-TOP, TOP).flatten(-2)[..., :C].to(FP8)
    return q.contiguous().view(torch.uint8), s


def _encode_weights(w):
    """FP8 codes and 128 x 128 block scales of one expert's w [N, K]."""
    N, K = w.shape
    n, m = -(-N // BLK), -(-K // BLK)
    b = torch.nn.functional.pad(w.float(), (0, m * BLK - K, 0, n * BLK - N)).view(n, BLK, m, BLK)
    s = b.abs().amax((1, 3)) / TOP
    q = (b / s[:, None, :, None]).clamp(-TOP, TOP).view(n * BLK, m * BLK)[:N, :K].to(FP8)
    return q.contiguous().view(torch.uint8), s


def _tokens(T, C, g):
    """Activations with a few large channels, as the residual stream of a model has."""
    big = 1.0 + 15.0 * (torch.rand(C, generator=g, device="cuda") < 0.01)
    return (torch.randn(T, C, generator=g, device="cuda") * big).to(torch.bfloat16)


def _route(T, E, k, skew, g):
    """Expert offsets and source tokens of the T * k routed rows, in group order."""
    prior = -skew * torch.log(torch.arange(1, E + 1, device="cuda").float())
    ids = (torch.randn(T, E, generator=g, device="cuda") + prior).topk(k, dim=1).indices.flatten()
    order = torch.sort(ids, stable=True).indices
    off = torch.zeros(E + 1, dtype=torch.int32, device="cuda")
    counts = torch.bincount(ids, minlength=E)
    off[1:] = counts.cumsum(0)
    return off, (order // k).to(torch.int32), int(counts.max())


def _weights(E, N, K, g):
    q = torch.empty(E, N, K, dtype=torch.uint8, device="cuda")
    s = torch.empty(E, -(-N // BLK), -(-K // BLK), device="cuda")
    for e in range(E):
        q[e], s[e] = _encode_weights(0.02 * torch.randn(N, K, generator=g, device="cuda"))
    return q, s


def prepare(case, seed):
    g = _generator(seed)
    st = dict(case)
    dev = "cuda"
    if case["op"] == "quantize":
        x = _tokens(case["T"], case["K"], g)
        st["x"] = x if case["bf16"] else x.float() * (1.0 + 1e-3 * torch.rand(x.shape, generator=g, device=dev))
        st["q"] = torch.empty(x.shape, dtype=torch.uint8, device=dev)
        st["sf"] = torch.empty(case["T"], -(-case["K"] // BLK), device=dev)
        return st
    T, E, k = case["T"], case["E"], case["k"]
    if case["op"] == "balance":
        S = case["S"]
        st["logits"] = torch.randn(T, E, generator=g, device=dev) * 1.5
        st["ids"] = st["logits"].topk(k, dim=1).indices.to(torch.int32)
        cuts = torch.randint(0, T + 1, (S - 1,), generator=g, device=dev).sort().values
        off = torch.zeros(S + 1, dtype=torch.int32, device=dev)
        off[1:-1] = cuts
        off[-1] = T
        st["off"] = off if S > 1 else None
        st["mask"] = None
        if case["masked"]:
            keep = torch.rand(T, generator=g, device=dev) >= case["masked"]
            st["mask"] = keep.to(torch.uint8)
            st["logits"][~keep] = float("nan")  # a padded row holds whatever was there
        st["grad"] = 0.5 + torch.rand(1, generator=g, device=dev)
        st["w"] = st["dw"] = None
        if case["routed"]:
            st["w"] = torch.softmax(torch.gather(st["logits"], 1, st["ids"].long()), 1)
            st["dw"] = 1e-3 * torch.randn(T, k, generator=g, device=dev)
        st["counts"] = torch.empty(S, E, dtype=torch.int32, device=dev)
        st["coef"] = torch.empty(S, E, device=dev)
        st["loss"] = torch.empty(1, device=dev)
        st["dlogits"] = torch.empty(T, E, device=dev)
        return st
    N, K = case["N"], case["K"]
    st["off"], st["src"], st["cap"] = _route(T, E, k, case["skew"], g)
    R = st["R"] = T * k
    x = _tokens(T, K, g)
    if case["op"] == "product":
        st["a"], st["as"] = _encode(x)
        st["b"], st["bs"] = _weights(E, N, K, g)
        st["out"] = torch.empty(R, N, dtype=torch.bfloat16, device=dev)
    elif case["op"] == "experts":
        st["x"] = x
        st["w1"], st["w1s"] = _weights(E, 2 * N, K, g)
        st["w2"], st["w2s"] = _weights(E, K, N, g)
    else:
        st["x"] = x
        st["w"] = torch.empty(E, N, K, dtype=torch.bfloat16, device=dev)
        for e in range(E):
            st["w"][e] = 0.02 * torch.randn(N, K, generator=g, device=dev)
        st["dy"] = (1e-3 * torch.randn(R, N, generator=g, device=dev)).to(torch.bfloat16)
    return st


# ---- plain form -----------------------------------------------------------------------------

def _up(s, n, dim):
    return s.repeat_interleave(BLK, dim).narrow(dim, 0, n)


def _scale(amax):
    """amax / 448 rounded once to 32 bits (a quotient by a constant may be taken as a product)."""
    return (amax.double() / TOP).float()


def _codes(b, s):
    """E4M3 of b / s, the quotient rounded once to 32 bits: values next to a border go by it."""
    return torch.where(s > 0, (b.double() / s).float(), 0.0).clamp(-TOP, TOP).to(FP8)


def _quantized(x, dim):
    """(codes as values, scales) of x with one scale per 128 along dim (padded with zeros)."""
    n = x.shape[dim]
    m = -(-n // BLK)
    pad = list(x.shape)
    pad[dim] = m * BLK - n
    b = torch.cat([x.float(), x.new_zeros(pad, dtype=torch.float32)], dim).unflatten(dim, (m, BLK))
    s = _scale(b.abs().amax(dim + 1))
    q = _codes(b, s.unsqueeze(dim + 1))
    return q.flatten(dim, dim + 1).narrow(dim, 0, n), s


def _dequantized(x, dim):
    q, s = _quantized(x, dim)
    return q.float() * _up(s, x.shape[dim], dim)


def _expert_of(off, R):
    return torch.searchsorted(off[1:].contiguous(), torch.arange(R, device=off.device, dtype=torch.int32), right=True)


def _padded(a, off, cap):
    """The groups of a's rows as [E, cap, C], zero behind each group."""
    at = torch.arange(cap, device=a.device)
    rows = (off[:-1, None] + at).clamp(max=a.shape[0] - 1)
    return a[rows] * (at < (off[1:] - off[:-1])[:, None])[..., None]


def _product(a, w, off, cap):
    """y[p] = a[p] . w[expert of p]^T over [R, K] and [E, N, K], all 32 bits."""
    R = a.shape[0]
    y = torch.bmm(_padded(a, off, cap), w.transpose(1, 2).contiguous())
    e = _expert_of(off, R)
    return y[e, torch.arange(R, device=a.device) - off[e]]


def _plain(st):
    op = st["op"]
    if op == "quantize":
        return _quantized(st["x"], 1)
    if op == "balance":
        return _plain_balance(st)
    off, src, cap, N, K = st["off"], st["src"].long(), st["cap"], st["N"], st["K"]
    if op == "product":
        a = (st["a"].view(FP8).float() * _up(st["as"], K, 1))[src]
        if st["R"] <= min(st["E"], 32):  # few rows: only their experts' weights
            e = _expert_of(off, st["R"])
            w = st["b"][e].view(FP8).float() * _up(_up(st["bs"][e], N, 1), K, 2)
            return (w * a[:, None, :]).sum(-1).to(torch.bfloat16)
        w = st["b"].view(FP8).float() * _up(_up(st["bs"], N, 1), K, 2)
        return _product(a, w, off, cap).to(torch.bfloat16)
    if op == "experts":
        w1 = st["w1"].view(FP8).float() * _up(_up(st["w1s"], 2 * N, 1), K, 2)
        y = _product(_dequantized(st["x"], 1)[src], w1, off, cap)
        del w1
        gate, up = y[:, :N], y[:, N:]
        act = _dequantized(gate / (1.0 + torch.exp(-gate)) * up, 1)
        w2 = st["w2"].view(FP8).float() * _up(_up(st["w2s"], K, 1), N, 2)
        return _product(act, w2, off, cap).to(torch.bfloat16)
    x, w, dy = st["x"].float(), st["w"], st["dy"].float()
    E = st["E"]
    n, m = -(-N // BLK), -(-K // BLK)
    b = torch.nn.functional.pad(w.float(), (0, m * BLK - K, 0, n * BLK - N)).view(E, n, BLK, m, BLK)
    s = _scale(b.abs().amax((2, 4)))[:, :, None, :, None]
    w8 = (_codes(b, s).float() * s).view(E, n * BLK, m * BLK)[:, :N, :K]
    y = _product(_dequantized(x, 1)[src], w8, off, cap)
    dx = _product(_dequantized(dy, 1), w8.transpose(1, 2), off, cap)
    dw = torch.bmm(_dequantized(_padded(dy, off, cap), 1).transpose(1, 2).contiguous(), _dequantized(_padded(x[src], off, cap), 1))
    return {"y": y.to(torch.bfloat16), "dx": dx.to(torch.bfloat16), "dw": dw}


def _plain_balance(st):
    T, E, k, S = st["T"], st["E"], st["k"], st["S"]
    logits, dev = st["logits"], st["logits"].device
    keep = torch.ones(T, dtype=torch.bool, device=dev) if st["mask"] is None else st["mask"] != 0
    z = torch.where(keep[:, None], logits, 0.0)
    p = torch.exp(z - z.amax(1, keepdim=True))
    p = p / p.sum(1, keepdim=True) * keep[:, None]
    seq = torch.zeros(T, dtype=torch.long, device=dev) if st["off"] is None else _expert_of(st["off"], T)
    of = ((seq == torch.arange(S, device=dev)[:, None]) & keep).double()  # [S, T]
    n = of.sum(1, keepdim=True)
    chosen = torch.zeros(T, E, dtype=torch.double, device=dev).scatter_add(1, st["ids"].long(), torch.ones(T, k, dtype=torch.double, device=dev))
    counts, mass = of @ chosen, of @ p.double()
    coef = torch.where(n > 0, E * counts / (k * n * n * S), 0.0)
    loss = (coef * mass).sum().view(1)
    a = st["grad"] * coef.float()[seq]
    d = p * (a - (p * a).sum(1, keepdim=True))
    if st["routed"]:
        w = torch.where(keep[:, None], st["w"], 0.0)
        d = d.scatter_add(1, st["ids"].long(), w * (st["dw"] - (w * st["dw"]).sum(1, keepdim=True)))
    return {"loss": loss.float(), "counts": counts.to(torch.int32), "dlogits": d}


# ---- the library ----------------------------------------------------------------------------

def _own(st):
    import block_scaled_fp4_02_amd as moe
    op = st["op"]
    if op == "quantize":
        moe.moe_quantize_fp8(st["x"], st["q"], st["sf"])
        return st["q"].view(FP8), st["sf"]
    if op == "balance":
        moe.moe_balance_loss(st["logits"], st["ids"], st["counts"], st["coef"], st["loss"], st["off"], st["mask"])
        moe.moe_balance_loss_backward(st["logits"], st["coef"], st["grad"], st["dlogits"], st["off"], st["mask"],
                                      st["ids"] if st["routed"] else None, st["w"], st["dw"])
        return {"loss": st["loss"], "counts": st["counts"], "dlogits": st["dlogits"]}
    off, src, R = st["off"], st["src"], st["R"]
    if op == "product":
        moe.moe_grouped_gemm_fp8(moe.make_gemm_fp8_args(st["a"], st["as"], st["b"], st["bs"], off, R, moe.MOE_EPI_NONE,
                                                        st["out"], A_rows=src))
        return st["out"]
    if op == "experts":
        xq = moe.quantize_fp8_alloc(st["x"])
        act = moe.grouped_gemm_fp8_alloc(xq, moe.FP8Tensor(st["w1"], st["w1s"]), off, R, moe.MOE_EPI_SWIGLU_FP8, A_rows=src)
        return moe.grouped_gemm_fp8_alloc(act, moe.FP8Tensor(st["w2"], st["w2s"]), off, R)
    w, wt = moe.quantize_fp8_weights_alloc(st["w"], transposed=True)
    y = moe.grouped_gemm_fp8_alloc(moe.quantize_fp8_alloc(st["x"]), w, off, R, A_rows=src)
    dx = moe.grouped_gemm_fp8_alloc(moe.quantize_fp8_alloc(st["dy"]), wt, off, R)
    dw = moe.grouped_wgrad_fp8_alloc(moe.quantize_fp8_tokens_alloc(st["dy"], off, R),
                                     moe.quantize_fp8_tokens_alloc(st["x"], off, R, rows=src), off, R)
    return {"y": y, "dx": dx, "dw": dw}


def run(state):
    return _own(state) if own else _plain(state)


# ---- what a pass cannot do without ----------------------------------------------------------

def work(case):
    op, T = case["op"], case["T"]
    if op == "quantize":
        n = T * case["K"]
        return {"bytes": n * (3 if case["bf16"] else 5) + T * -(-case["K"] // BLK) * 4, "flops": 3 * n}
    E, k = case["E"], case["k"]
    if op == "balance":
        rows = T * E * 4
        extra = T * k * 4 * (2 if case["routed"] else 0) + (T if case["masked"] else 0)
        return {"bytes": 2 * rows + T * k * 4 + extra + case["S"] * E * 4, "flops": 12 * T * E}
    N, K, R = case["N"], case["K"], T * k
    hit = E * (1.0 - (1.0 - k / E) ** T) if E > k else E  # experts that get a row
    if op == "product":
        return {"bytes": hit * N * K + min(T, R) * K + R * N * 2, "flops": 2 * R * N * K}
    if op == "experts":
        return {"bytes": 3 * hit * N * K + T * K * 2 + R * K * 2, "flops": 6 * R * N * K}
    return {"bytes": E * N * K * (2 + 4) + T * K * 2 + R * N * 2 + R * (N + K) * 2, "flops": 6 * R * N * K}


# ---- the definition in 64 bits --------------------------------------------------------------

def _value(code_bytes):
    """E4M3 values of code bytes, from the format: sign, 4 exponent bits of bias 7, 3 mantissa bits."""
    c = torch.arange(256, device=code_bytes.device)
    e, m = (c >> 3) & 15, (c & 7).double()
    v = torch.where(e == 0, m * 2.0 ** -9, (1 + m / 8) * 2.0 ** (e.double() - 7))
    v = torch.where((c & 127) == 127, float("nan"), v) * torch.where(c >= 128, -1.0, 1.0)
    return v[code_bytes.long()]


def _round_e4m3(u):
    """Nearest E4M3 value to u, |u| <= 448, ties to the even one."""
    _, e = torch.frexp(u)
    step = torch.ldexp(torch.ones_like(u), (e - 1).clamp(min=-6) - 3)
    return torch.round(u / step) * step


def _stored(x, dim):
    """What the stored codes and scales of x stand for: the scale amax / 448 and the quotients by
    it are each rounded to binary32, as the definition says, the quotient then to E4M3."""
    parts, scales = [], []
    for b in x.split(BLK, dim):
        s = (b.abs().amax(dim, keepdim=True) / TOP).float().double()
        u = torch.where(s > 0, b / s, 0.0).float().double().clamp(-TOP, TOP)
        parts.append(_round_e4m3(u))
        scales.append(s)
    return torch.cat(parts, dim), torch.cat(scales, dim)


def _spread(s, n, dim):
    return s.index_select(dim, torch.arange(n, device=s.device) // BLK)


def _stored_value(x, dim):
    v, s = _stored(x, dim)
    return v * _spread(s, x.shape[dim], dim)


def exact(case, seed):
    st = prepare(case, seed)
    op = case["op"]
    if op == "quantize":
        v, s = _stored(st["x"].double(), 1)
        return v, s
    if op == "balance":
        return _exact_balance(st)
    N, K = case["N"], case["K"]
    bounds, src = st["off"].tolist(), st["src"].long()
    groups = list(zip(range(case["E"]), bounds, bounds[1:]))
    if op == "product":
        y = torch.empty(st["R"], N, dtype=torch.double, device="cuda")
        a = _value(st["a"]) * _spread(st["as"].double(), K, 1)
        for e, lo, hi in groups:
            if hi > lo:
                y[lo:hi] = a[src[lo:hi]] @ (_value(st["b"][e]) * _spread(_spread(st["bs"][e].double(), N, 0), K, 1)).T
        return y
    x = st["x"].double()
    if op == "experts":
        y = torch.empty(st["R"], K, dtype=torch.double, device="cuda")
        a = _stored_value(x, 1)
        for e, lo, hi in groups:
            if hi > lo:
                h = a[src[lo:hi]] @ (_value(st["w1"][e]) * _spread(_spread(st["w1s"][e].double(), 2 * N, 0), K, 1)).T
                act = _stored_value(h[:, :N] * torch.sigmoid(h[:, :N]) * h[:, N:], 1)
                y[lo:hi] = act @ (_value(st["w2"][e]) * _spread(_spread(st["w2s"][e].double(), K, 0), N, 1)).T
        return y
    dy = st["dy"].double()
    y = torch.empty(st["R"], N, dtype=torch.double, device="cuda")
    dx = torch.empty(st["R"], K, dtype=torch.double, device="cuda")
    dw = torch.zeros(case["E"], N, K, dtype=torch.double, device="cuda")
    a, d = _stored_value(x, 1), _stored_value(dy, 1)
    for e, lo, hi in groups:
        if hi > lo:
            w = st["w"][e].double()
            peak = torch.stack([c.abs().amax(1) for c in w.split(BLK, 1)], 1)
            s = torch.stack([r.amax(0) for r in peak.split(BLK, 0)], 0) / TOP
            s = _spread(_spread(s.float().double(), N, 0), K, 1)
            w = _round_e4m3(torch.where(s > 0, w / s, 0.0).float().double().clamp(-TOP, TOP)) * s
            y[lo:hi] = a[src[lo:hi]] @ w.T
            dx[lo:hi] = d[lo:hi] @ w
            dw[e] = _stored_value(dy[lo:hi], 0).T @ _stored_value(x[src[lo:hi]], 0)
    return {"y": y, "dx": dx, "dw": dw}


def _exact_balance(st):
    T, E, k, S = st["T"], st["E"], st["k"], st["S"]
    bounds = [0, T] if st["off"] is None else st["off"].tolist()
    keep = torch.ones(T, dtype=torch.bool, device="cuda") if st["mask"] is None else st["mask"].bool()
    loss = torch.zeros(1, dtype=torch.double, device="cuda")
    counts = torch.zeros(S, E, dtype=torch.int32, device="cuda")
    d = torch.zeros(T, E, dtype=torch.double, device="cuda")
    for s, (lo, hi) in enumerate(zip(bounds, bounds[1:])):
        rows = torch.arange(lo, hi, device="cuda")[keep[lo:hi]]
        n = rows.numel()
        if n == 0:
            continue
        ids = st["ids"][rows].long()
        counts[s] = torch.bincount(ids.flatten(), minlength=E)
        p = torch.softmax(st["logits"][rows].double(), 1)
        f = counts[s].double() * E / (k * n)
        loss += (f * p.mean(0)).sum() / S
        a = st["grad"].double() * f / (n * S)
        d[rows] = p * (a - (p @ a)[:, None])
        if st["routed"]:
            w, dw = st["w"][rows].double(), st["dw"][rows].double()
            own_part = torch.zeros(n, E, dtype=torch.double, device="cuda")
            own_part.scatter_add_(1, ids, w * (dw - (w * dw).sum(1, keepdim=True)))
            d[rows] += own_part
    return {"loss": loss, "counts": counts, "dlogits": d}
