"""Measured cases of the scored router, the FP8 grouped products and the SwiGLU with 8-bit activation checkpoints.

``own`` chooses between the plain form (elementary torch operations) and the framework's calls.  The shapes are
those of the framework's own workloads: d = 7168, inter = 2048, E = 256 or 384 experts, top-8, batches of 64
(decode) and 8192 (prefill) tokens, with odd batch sizes beside them.
"""
import math

import numpy as np
import torch

own = False

DEV = "cuda"
BLOCK = 128          # values that share one scale
E4M3_MAX = 448.0


# ------------------------------------------------------------------ cases

def listed():
    return [
        # router of one decode step: softmax scores, BF16 logits, launch latency counts
        dict(name="route_decode", op="route", T=64, E=384, k=8, score="softmax", n_group=1, topk_group=1, group_top=1,
             bias=False, renorm=True, scale=1.0, dtype="bf16"),
        # router of a prefill batch: sigmoid scores, balance bias, 4 of 8 groups by their two best
        dict(name="route_prefill", op="route", T=8192, E=256, k=8, score="sigmoid", n_group=8, topk_group=4, group_top=2,
             bias=True, renorm=True, scale=2.5, dtype="fp32"),
        # router gradient of a training batch, nonzero at the kept experts only
        dict(name="route_bwd_sigmoid", op="route_bwd", T=8192, E=256, k=8, score="sigmoid", renorm=True, scale=2.5,
             dtype="fp32"),
        # router gradient that reaches every expert (softmax kept as it is)
        dict(name="route_bwd_softmax", op="route_bwd", T=1001, E=384, k=8, score="softmax", renorm=False, scale=1.0,
             dtype="bf16"),
        # gate_up product of a decode batch with few, uneven experts: streams their weights
        dict(name="gemm_decode", op="gemm", T=64, E=384, k=8, N=4096, K=7168, trans=False, sorted=False, given="bf16",
             wscale="e8m0", zipf=1.2),
        # gate_up product of a prefill batch: about 256 rows an expert
        dict(name="gemm_prefill", op="gemm", T=8192, E=256, k=8, N=4096, K=7168, trans=False, sorted=False, given="bf16",
             wscale="e8m0", zipf=0.0),
        # input gradient of the down projection, an odd batch, weights whose scales are any fp32 number
        dict(name="gemm_t_down", op="gemm", T=1001, E=64, k=8, N=7168, K=2048, trans=True, sorted=False, given="bf16",
             wscale="fp32", zipf=0.0),
        # input gradient of gate_up on the gradient that the SwiGLU backward left in 8 bits
        dict(name="gemm_t_gate_up", op="gemm", T=8192, E=256, k=8, N=4096, K=7168, trans=True, sorted=True, given="fp8",
             wscale="e8m0", zipf=0.0),
        # SwiGLU of a decode-sized batch, quantised for the down projection
        dict(name="swiglu_small", op="swiglu", T=64, k=8, inter=2048),
        # SwiGLU of a training batch with its 8-bit checkpoint
        dict(name="swiglu_prefill", op="swiglu", T=8192, k=8, inter=2048),
        # backward from the checkpoint, BF16 gradient (for 4-bit weights), an odd batch
        dict(name="swiglu_bwd_bf16", op="swiglu_bwd", T=1001, k=8, inter=2048, out="bf16"),
        # backward from the checkpoint, gradient in 8 bits for the FP8 product
        dict(name="swiglu_bwd_fp8", op="swiglu_bwd", T=8192, k=8, inter=2048, out="fp8"),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["route", "route_bwd", "gemm", "gemm", "swiglu", "swiglu_bwd"])
    T = _log_int(rng, 1, 8192)
    if op in ("route", "route_bwd"):
        n_group = rng.choice([1, 1, 4, 8])
        E = n_group * rng.randint(8, 384 // n_group)
        topk_group = rng.randint(max(1, n_group // 2), n_group)
        c = dict(op=op, T=T, E=E, k=rng.randint(1, 8), score=rng.choice(["softmax", "sigmoid"]),
                 renorm=rng.random() < 0.7, scale=rng.choice([1.0, 2.5]), dtype=rng.choice(["fp32", "bf16"]))
        if op == "route":
            c.update(n_group=n_group, topk_group=topk_group, group_top=rng.choice([1, 2]), bias=rng.random() < 0.7)
        return c
    if op == "gemm":
        zipf = rng.choice([0.0, 1.2])
        if zipf:
            T = min(T, 512)      # uneven routing at decode sizes
        E = _log_int(rng, 8, 256)
        N, K = 64 * _log_int(rng, 4, 64), 128 * _log_int(rng, 2, 56)
        trans = rng.random() < 0.5
        return dict(op=op, T=T, E=E, k=rng.randint(1, 8), N=N, K=K, trans=trans, sorted=trans and rng.random() < 0.5,
                    given=rng.choice(["bf16", "fp8"]), wscale=rng.choice(["e8m0", "fp32"]), zipf=zipf)
    c = dict(op=op, T=T, k=rng.randint(1, 8), inter=128 * rng.randint(1, 16))
    if op == "swiglu_bwd":
        c["out"] = rng.choice(["bf16", "fp8"])
    return c


# ------------------------------------------------------------------ inputs

def _generator(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return g


def _normal(g, *shape, std=1.0, dtype=torch.bfloat16):
    return (torch.randn(*shape, generator=g, device=DEV) * std).to(dtype)


def _scale_exponent(amax):
    """e, the least whole number with amax <= 448 * 2^e, at least -127; 0 where amax is 0."""
    m, ex = torch.frexp(amax)
    e = torch.where(m <= 0.875, ex - 9, ex - 8).clamp(min=-127)
    return torch.where(amax > 0, e, torch.zeros_like(e))


def _power(e):
    """2^e in 32 bits, -126 <= e <= 127, put together from its bits."""
    return ((e + 127).to(torch.int32) << 23).view(torch.float32)


def _quantize(x):
    """Rows of x in blocks of 128: (e4m3 codes, E8M0 scales) as fp8_quantize defines them; a last block may be short."""
    rows, cols = x.shape
    x = x.float()
    nb = -(-cols // BLOCK)
    if nb * BLOCK != cols:
        x = torch.nn.functional.pad(x, (0, nb * BLOCK - cols))
    x = x.view(rows, nb, BLOCK)
    e = _scale_exponent(x.abs().amax(dim=2))
    codes = (x * _power(-e)[:, :, None]).to(torch.float8_e4m3fn)
    codes = codes.view(rows, nb * BLOCK)[:, :cols].contiguous()
    return codes, (e + 127).to(torch.uint8).view(torch.float8_e8m0fnu)


def _dequantize(codes, scales):
    rows, cols = codes.shape
    s = scales.float().repeat_interleave(BLOCK, dim=1)[:, :cols]
    return codes.float() * s


def _weights(g, E, N, K, wscale):
    """Codes [E, N, K] and scales [E, ceil(N/128), K/128] of normal weights."""
    nb, kb = -(-N // BLOCK), K // BLOCK
    codes = torch.empty((E, N, K), dtype=torch.float8_e4m3fn, device=DEV)
    scales = torch.empty((E, nb, kb), dtype=torch.float32 if wscale == "fp32" else torch.uint8, device=DEV)
    step = max(1, (1 << 28) // (N * K))
    for e0 in range(0, E, step):
        n = min(step, E - e0)
        w = torch.zeros((n, nb * BLOCK, K), device=DEV)
        w[:, :N] = torch.randn(n, N, K, generator=g, device=DEV) * 0.02
        # experts differ in size, as trained ones do
        w *= torch.exp2(torch.randn(n, nb, 1, kb, 1, generator=g, device=DEV)).expand(n, nb, BLOCK, kb, BLOCK).reshape(w.shape)
        blocks = w.view(n, nb, BLOCK, kb, BLOCK)
        amax = blocks.abs().amax(dim=(2, 4))
        if wscale == "fp32":
            s = amax / E4M3_MAX
            scales[e0:e0 + n] = s
        else:
            ex = _scale_exponent(amax)
            s = _power(ex)
            scales[e0:e0 + n] = (ex + 127).to(torch.uint8)
        q = (blocks / s[:, :, None, :, None]).view(n, nb * BLOCK, K)[:, :N]
        codes[e0:e0 + n] = q.clamp(-E4M3_MAX, E4M3_MAX).to(torch.float8_e4m3fn)
    return codes, scales if wscale == "fp32" else scales.view(torch.float8_e8m0fnu)


def _plan(ids, E):
    """The permutation of the pairs by expert, as expert_permute lays it out."""
    flat = ids.reshape(-1).long()
    P = flat.numel()
    order = torch.argsort(flat, stable=True)
    counts = torch.bincount(flat, minlength=E)
    offsets = torch.zeros(E + 1, dtype=torch.int64, device=DEV)
    offsets[1:] = torch.cumsum(counts, 0)
    inv = torch.empty(P, dtype=torch.int64, device=DEV)
    inv[order] = torch.arange(P, device=DEV)
    live = torch.nonzero(counts).flatten()
    active = torch.full((E,), -1, dtype=torch.int64, device=DEV)
    active[:live.numel()] = live
    i32 = lambda t: t.to(torch.int32).contiguous()  # noqa: E731
    return dict(counts=i32(counts), offsets=i32(offsets), perm=i32(order), inv_perm=i32(inv), active=i32(active),
                n_active=torch.tensor([live.numel()], dtype=torch.int32, device=DEV))


def _popularity(E, zipf, rng):
    return -zipf * np.log(1.0 + rng.permutation(E)) if zipf > 0 else np.zeros(E)


def prepare(case, seed):
    g = _generator(seed)
    op = case["op"]
    st = dict(case=case, op=op)
    if op in ("route", "route_bwd"):
        T, E, k = case["T"], case["E"], case["k"]
        dt = torch.float32 if case["dtype"] == "fp32" else torch.bfloat16
        st["logits"] = _normal(g, T, E, std=1.5, dtype=dt)
        st["bias"] = None
        if op == "route":
            if case["bias"]:
                st["bias"] = _normal(g, E, std=0.05, dtype=torch.float32)
        else:
            st["ids"] = torch.topk(st["logits"].float(), k, dim=1).indices.to(torch.int32)
            st["dgates"] = _normal(g, T, k, dtype=torch.float32)
        return st
    T, k = case["T"], case["k"]
    P = T * k
    if op == "gemm":
        E, N, K = case["E"], case["N"], case["K"]
        pop = _popularity(E, case["zipf"], np.random.RandomState(seed))
        logits = _normal(g, T, E, dtype=torch.float32) + torch.tensor(pop, dtype=torch.float32, device=DEV)
        st["plan"] = _plan(torch.topk(logits, k, dim=1).indices, E)
        st["w"], st["w_scales"] = _weights(g, E, N, K, case["wscale"])
        a = _normal(g, P if case["sorted"] else T, N if case["trans"] else K)
        if case["given"] == "fp8":
            st["a"], st["a_scales"] = _quantize(a)
        else:
            st["a"], st["a_scales"] = a, None
        st["live"] = int(st["plan"]["n_active"])
        st["most"] = int(st["plan"]["counts"].max())
        return st
    ids = torch.argsort(torch.rand(T, 4 * k, generator=g, device=DEV), dim=1)[:, :k]
    inter = case["inter"]
    h = _normal(g, P, 2 * inter, std=1.5)
    if op == "swiglu":
        st["h"] = h
        return st
    st["plan"] = _plan(ids, 4 * k)
    st["h8"], st["h8_scales"] = _quantize(h)
    st["da"] = _normal(g, P, inter)
    st["gates"] = torch.softmax(torch.randn(T, k, generator=g, device=DEV), dim=1)
    return st


# ------------------------------------------------------------------ plain forms

def _choose(c, n_group, topk_group, group_top, k):
    """The k best of each row of c, from its best groups; equal values in the order of their ids."""
    T, E = c.shape
    if topk_group < n_group:
        per = c.view(T, n_group, E // n_group)
        best = torch.sort(per, dim=2, descending=True).values[:, :, :group_top].sum(dim=2)
        kept = torch.sort(best, dim=1, descending=True, stable=True).indices[:, :topk_group]
        stays = torch.zeros((T, n_group), dtype=torch.bool, device=c.device).scatter_(1, kept, True)
        c = c.masked_fill(~stays.repeat_interleave(E // n_group, dim=1), -math.inf)
    return torch.sort(c, dim=1, descending=True, stable=True).indices[:, :k]


def _scores(logits, score):
    l = logits.double()
    if score == "sigmoid":
        return 1.0 / (1.0 + torch.exp(-l))
    p = torch.exp(l - l.amax(dim=1, keepdim=True))
    return p / p.sum(dim=1, keepdim=True)


def _route(st):
    c = st["case"]
    s = _scores(st["logits"], c["score"])           # 64 bits: the choice must not hang on the rounding of a score
    choice = s if st["bias"] is None else s + st["bias"].double()
    ids = _choose(choice, c["n_group"], c["topk_group"], c["group_top"], c["k"])
    w = torch.gather(s, 1, ids)
    if c["renorm"]:
        w = w / w.sum(dim=1, keepdim=True)
    return dict(ids=ids.to(torch.int32), gates=(w * c["scale"]).float())


def _route_bwd(st):
    c = st["case"]
    l, dg = st["logits"].float(), st["dgates"]
    ids = st["ids"].long()
    if c["score"] == "sigmoid":
        kept = torch.sigmoid(torch.gather(l, 1, ids))
        slope = kept * (1 - kept)
    else:
        p = torch.exp(l - l.amax(dim=1, keepdim=True))
        p = p / p.sum(dim=1, keepdim=True)
        kept = torch.gather(p, 1, ids)
    if c["renorm"]:
        total = kept.sum(dim=1, keepdim=True)
        w = kept / total
        inner = dg - (dg * w).sum(dim=1, keepdim=True)
        v = inner * slope / total if c["score"] == "sigmoid" else inner * w
        out = torch.zeros_like(l).scatter_add_(1, ids, v)
    elif c["score"] == "sigmoid":
        out = torch.zeros_like(l).scatter_add_(1, ids, dg * slope)
    else:
        out = -p * (dg * kept).sum(dim=1, keepdim=True)
        out = out.scatter_add(1, ids, dg * kept)
    return (out * c["scale"]).to(st["logits"].dtype)


def _gemm(st):
    c = st["case"]
    codes, scales = (st["a"], st["a_scales"]) if c["given"] == "fp8" else _quantize(st["a"])
    a = _dequantize(codes, scales)
    plan, N, K, k = st["plan"], c["N"], c["K"], c["k"]
    live, most, P = st["live"], st["most"], c["T"] * k
    act = plan["active"][:live].long()
    first, count = plan["offsets"][:-1][act].long(), plan["counts"][act].long()
    # every live expert's rows, padded to the longest
    at = torch.arange(most, device=DEV)[None, :]
    row = first[:, None] + torch.minimum(at, count[:, None] - 1)
    src = row if c["sorted"] else plan["perm"][row].long() // k
    xs = a[src.reshape(-1)].view(live, most, a.shape[1])
    whole = live == c["E"]
    w = (st["w"] if whole else st["w"].view(torch.uint8)[act].view(torch.float8_e4m3fn)).float()
    s = st["w_scales"].float()[act]
    nb = s.shape[1]
    if nb * BLOCK == N:
        w.view(live, nb, BLOCK, K // BLOCK, BLOCK).mul_(s[:, :, None, :, None])
    else:
        w.mul_(s.repeat_interleave(BLOCK, 1)[:, :N].repeat_interleave(BLOCK, 2))
    y = torch.bmm(xs, w) if c["trans"] else torch.bmm(w, xs.transpose(1, 2).contiguous()).transpose(1, 2)
    keep = at < count[:, None]
    out = torch.empty((P, K if c["trans"] else N), dtype=torch.bfloat16, device=DEV)
    out[row[keep]] = y[keep].to(torch.bfloat16)
    return out


def _swiglu(st):
    I = st["case"]["inter"]
    h = st["h"]
    gate, up = h[:, :I].float(), h[:, I:].float()
    a, a_scales = _quantize(gate / (1 + torch.exp(-gate)) * up)
    h8, h8_scales = _quantize(h)
    return dict(a=a, a_scales=a_scales, h=h8, h_scales=h8_scales)


def _swiglu_bwd(st):
    c = st["case"]
    I = c["inter"]
    h = _dequantize(st["h8"], st["h8_scales"])
    gate, up, da = h[:, :I], h[:, I:], st["da"].float()
    sig = 1 / (1 + torch.exp(-gate))
    silu = gate * sig
    pair = st["plan"]["perm"].long()
    dgates = torch.zeros(c["T"] * c["k"], device=DEV)
    dgates[pair] = (da * silu * up).double().sum(dim=1).float()
    d = da * st["gates"].reshape(-1)[pair][:, None]
    dh = torch.cat([d * up * sig * (1 + gate * (1 - sig)), d * silu], dim=1)
    dgates = dgates.view(c["T"], c["k"])
    if c["out"] == "bf16":
        return dict(dh=dh.to(torch.bfloat16), dgates=dgates)
    dh8, scales = _quantize(dh)
    return dict(dh=dh8, dh_scales=scales, dgates=dgates)


# ------------------------------------------------------------------ the framework's calls

def _perm(plan, qgg):
    return qgg.Perm(**{n: plan[n] for n in ("counts", "offsets", "perm", "inv_perm", "active", "n_active")})


def _own(st):
    import quantized_grouped_gemm_amd as qgg
    c, op = st["case"], st["op"]
    if op == "route":
        ids, gates = qgg.moe_route_scored(st["logits"], c["k"], score=c["score"], bias=st["bias"], n_group=c["n_group"],
                                          topk_group=c["topk_group"], group_top=c["group_top"], renorm=c["renorm"],
                                          scale=c["scale"])
        return dict(ids=ids, gates=gates)
    if op == "route_bwd":
        return qgg.moe_route_scored_bwd(st["logits"], st["ids"], st["dgates"], score=c["score"], renorm=c["renorm"],
                                        scale=c["scale"])
    if op == "gemm":
        a, s = (st["a"], st["a_scales"]) if c["given"] == "fp8" else qgg.fp8_quantize(st["a"])
        flags = (qgg.A_SORTED if c["sorted"] else qgg.A_TOKENS) | (qgg.TRANSPOSE_W if c["trans"] else 0)
        return qgg.fp8_grouped_gemm(qgg.Fp8Weight(st["w"], st["w_scales"]), a, s, _perm(st["plan"], qgg), c["T"], c["k"],
                                    flags=flags)
    if op == "swiglu":
        r = qgg.swiglu_fp8(st["h"], want=("a8", "h8"))
        return dict(a=r["a8"], a_scales=r["a8_scales"], h=r["h8"], h_scales=r["h8_scales"])
    kind = "dh" if c["out"] == "bf16" else "dh8"
    r = qgg.swiglu_fp8_bwd(st["da"], st["h8"], st["h8_scales"], st["gates"], _perm(st["plan"], qgg), want=(kind, "dgates"))
    if kind == "dh":
        return dict(dh=r["dh"], dgates=r["dgates"])
    return dict(dh=r["dh8"], dh_scales=r["dh8_scales"], dgates=r["dgates"])


def run(state):
    if own:
        return _own(state)
    return dict(route=_route, route_bwd=_route_bwd, gemm=_gemm, swiglu=_swiglu, swiglu_bwd=_swiglu_bwd)[state["op"]](state)


# ------------------------------------------------------------------ bytes and operations

def _live_experts(c):
    """How many experts a batch of this routing reaches, from one simulated batch."""
    rng = np.random.RandomState(7)
    logits = rng.randn(c["T"], c["E"]) + _popularity(c["E"], c["zipf"], rng)
    return int(np.unique(np.argpartition(-logits, c["k"] - 1, axis=1)[:, :c["k"]]).size)


def work(case):
    c, op, T, k = case, case["op"], case["T"], case["k"]
    P = T * k
    if op == "route":
        size = 4 if c["dtype"] == "fp32" else 2
        return dict(bytes=T * c["E"] * size + (4 * c["E"] if c["bias"] else 0) + P * 8, flops=8 * T * c["E"])
    if op == "route_bwd":
        size = 4 if c["dtype"] == "fp32" else 2
        dense = c["score"] == "softmax" and not c["renorm"]
        return dict(bytes=(T * c["E"] if dense else P) * size + P * 8 + T * c["E"] * size,
                    flops=(8 * T * c["E"] if dense else 16 * P))
    if op == "gemm":
        N, K = c["N"], c["K"]
        rows, width, out = P if c["sorted"] else T, N if c["trans"] else K, K if c["trans"] else N
        a = rows * width * (2 if c["given"] == "bf16" else 1 + 1 / BLOCK)
        w = _live_experts(c) * (N * K + -(-N // BLOCK) * (K // BLOCK) * (4 if c["wscale"] == "fp32" else 1))
        return dict(bytes=int(a + w + P * out * 2), flops=2 * P * N * K)
    n = P * c["inter"]
    if op == "swiglu":
        return dict(bytes=int(n * 4 + n * 3 * (1 + 1 / BLOCK)), flops=20 * n)
    out = 4 * n if c["out"] == "bf16" else 2 * n * (1 + 1 / BLOCK)
    return dict(bytes=int(2 * n + 2 * n * (1 + 1 / BLOCK) + out + P * 12), flops=40 * n)


# ------------------------------------------------------------------ 64-bit results

def _round_e4m3(v):
    """v (64 bits, at most 448 in size) on the e4m3 grid: three mantissa bits, least exponent -6, ties to even."""
    _, ex = torch.frexp(v)
    step = torch.exp2((ex - 1).clamp(min=-6).double() - 3)
    return torch.round(v / step) * step


def _exact_quantize(x):
    rows, cols = x.shape
    nb = -(-cols // BLOCK)
    codes, scales = torch.zeros_like(x), torch.ones((rows, nb), dtype=torch.float64, device=x.device)
    for b in range(nb):
        part = x[:, b * BLOCK:(b + 1) * BLOCK]
        top = part.abs().amax(dim=1)
        e = torch.ceil(torch.log2(torch.where(top > 0, top, 448.0 * torch.ones_like(top)) / 448.0) - 1e-14).clamp(min=-127)
        scales[:, b] = torch.exp2(e)
        codes[:, b * BLOCK:(b + 1) * BLOCK] = _round_e4m3(part / scales[:, b:b + 1])
    return codes, scales


def _exact_value(codes, scales):
    out = codes.double()
    for b in range(scales.shape[1]):
        out[:, b * BLOCK:(b + 1) * BLOCK] *= scales[:, b:b + 1].double()
    return out


def _exact_route(c, st):
    l = st["logits"].double().cpu().numpy()
    T, E = l.shape
    if c["score"] == "sigmoid":
        s = 1 / (1 + np.exp(-l))
    else:
        s = np.exp(l - l.max(axis=1, keepdims=True))
        s /= s.sum(axis=1, keepdims=True)
    choice = s + (0.0 if st["bias"] is None else st["bias"].double().cpu().numpy())
    size = E // c["n_group"]
    ids = np.empty((T, c["k"]), np.int64)
    for t in range(T):
        v = choice[t]
        pool = np.arange(E)
        if c["topk_group"] < c["n_group"]:
            best = [np.sort(v[j * size:(j + 1) * size])[::-1][:c["group_top"]].sum() for j in range(c["n_group"])]
            kept = sorted(range(c["n_group"]), key=lambda j: (-best[j], j))[:c["topk_group"]]
            pool = np.concatenate([np.arange(j * size, (j + 1) * size) for j in sorted(kept)])
        ids[t] = pool[np.argsort(-v[pool], kind="stable")[:c["k"]]]
    w = np.take_along_axis(s, ids, 1)
    if c["renorm"]:
        w = w / w.sum(axis=1, keepdims=True)
    return dict(ids=torch.from_numpy(ids.astype(np.int32)), gates=torch.from_numpy(w * c["scale"]))


def _exact_route_bwd(c, st):
    """By the product rule, from the Jacobian of the kept gates with respect to their scores."""
    l, dg, ids = st["logits"].double(), st["dgates"].double(), st["ids"].long()
    s = torch.special.expit(l) if c["score"] == "sigmoid" else torch.softmax(l, 1)
    u = torch.gather(s, 1, ids)
    du = dg * c["scale"]
    if c["renorm"]:
        total = u.sum(1, keepdim=True)
        du = (du * total - (du * u).sum(1, keepdim=True)) / total ** 2
    ds = torch.zeros_like(s).scatter_add_(1, ids, du)
    if c["score"] == "sigmoid":
        return ds * s * (1 - s)
    return s * (ds - (ds * s).sum(1, keepdim=True))


def _exact_gemm(c, st):
    if c["given"] == "fp8":
        a = _exact_value(st["a"], st["a_scales"])
    else:
        a = _exact_value(*_exact_quantize(st["a"].double()))
    plan, N, K = st["plan"], c["N"], c["K"]
    off = plan["offsets"].tolist()
    out = torch.zeros((c["T"] * c["k"], K if c["trans"] else N), dtype=torch.float64, device=a.device)
    for e in range(c["E"]):
        if off[e] == off[e + 1]:
            continue
        w = st["w"][e].double()
        s = st["w_scales"][e].double()
        for b in range(s.shape[0]):
            w[b * BLOCK:(b + 1) * BLOCK] *= s[b].repeat_interleave(BLOCK)
        rows = torch.arange(off[e], off[e + 1], device=a.device)
        src = rows if c["sorted"] else plan["perm"][rows].long() // c["k"]
        out[rows] = a[src] @ (w if c["trans"] else w.t())
    return out


def _exact_swiglu(c, st):
    h = st["h"].double()
    gate, up = h[:, :c["inter"]], h[:, c["inter"]:]
    a, a_scales = _exact_quantize(gate * torch.special.expit(gate) * up)
    h8, h_scales = _exact_quantize(h)
    return dict(a=a, a_scales=a_scales, h=h8, h_scales=h_scales)


def _exact_swiglu_bwd(c, st):
    I = c["inter"]
    h = _exact_value(st["h8"], st["h8_scales"])
    gate, up = h[:, :I], h[:, I:]
    pair = st["plan"]["perm"].long()
    f = torch.special.expit(gate)
    raw = st["da"].double()
    dgates = torch.zeros(c["T"] * c["k"], dtype=torch.float64, device=h.device)
    dgates[pair] = (raw * gate * f * up).sum(1)
    d = raw * st["gates"].double().reshape(-1)[pair].unsqueeze(1)
    dh = torch.empty_like(h)
    dh[:, :I] = d * up * (f + gate * f * (1 - f))
    dh[:, I:] = d * gate * f
    dgates = dgates.view(c["T"], c["k"])
    if c["out"] == "bf16":
        return dict(dh=dh, dgates=dgates)
    dh8, scales = _exact_quantize(dh)
    return dict(dh=dh8, dh_scales=scales, dgates=dgates)


def exact(case, seed):
    st = prepare(case, seed)
    return dict(route=_exact_route, route_bwd=_exact_route_bwd, gemm=_exact_gemm, swiglu=_exact_swiglu,
                swiglu_bwd=_exact_swiglu_bwd)[case["op"]](case, st)
