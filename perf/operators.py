"""The operators around the FP8 linear layer of a rollout or training step: what
is measured, and their plain forms.

Residual addition with RMSNorm and 1x128 quantization (forward and backward),
rotary positions (forward, backward, and fused with the FP8 KV-cache write),
block tables and slot maps of a paged KV cache, and sampling.  ``run`` computes
them with elementary torch operations where ``own`` is false, and calls the
package's entry points where it is true.  ``exact`` is the same definition in
64 bits, written apart.
"""
import math

import torch

own = False

DEV = "cuda"
BF16, F32, F64, I32, I64, U8, F8 = (torch.bfloat16, torch.float32, torch.float64, torch.int32,
                                    torch.int64, torch.uint8, torch.float8_e4m3fn)
NEG = float("-inf")


# --------------------------------------------------------------------------
# cases
# --------------------------------------------------------------------------

def listed():
    return [
        # the residual stream between two layers of the 8B-shaped model, 16 sequences decoding
        dict(name="norm_decode", op="norm", M=16, K=4096, eps=1e-5),
        # the same of the 32B-shaped model over a training step's 16384 tokens
        dict(name="norm_train32b", op="norm", M=16384, K=5120, eps=1e-6),
        # its backward in the 8B-shaped layer: gradients of q, k and v, and of the residual stream
        dict(name="norm_bwd_train8b", op="norm_bwd", M=8192, K=4096, n_dy=3, dres=True),
        # a ragged batch's MLP norm at the end of the stream: gradients of gate and up only
        dict(name="norm_bwd_ragged", op="norm_bwd", M=1537, K=5120, n_dy=2, dres=False),
        # training step of the 8B-shaped layer: q and k of 8192 tokens, frequencies scaled for long contexts
        dict(name="rope_train8b", op="rope", T=8192, Hq=32, Hk=8, D=128, R=128, layout="half",
             scaling="wavelength", factor=8.0, backward=False, packed=False, start=0),
        # backward of half-rotated heads with interleaved pairs, far into a long context, odd token count
        dict(name="rope_bwd_part", op="rope", T=4099, Hq=64, Hk=8, D=128, R=64,
             layout="interleaved", scaling="linear", factor=4.0, backward=True, packed=True,
             start=1000000),
        # 64 sequences decoding: rotate q and k, write k and v to the FP8 cache
        dict(name="rope_kv_decode", op="rope_kv", T=64, Hq=32, Hk=8, D=128, R=128, layout="half",
             scaling="wavelength", factor=8.0, packed=True, S=65536, start=5000),
        # a 16384-token prefill of the 32B-shaped model's heads
        dict(name="rope_kv_prefill", op="rope_kv", T=16384, Hq=64, Hk=8, D=128, R=128,
             layout="half", scaling="none", factor=1.0, packed=False, S=32768, start=0),
        # one decoding step of 256 requests
        dict(name="slots_decode", op="slots", B=256, most_added=1, most_cached=8192, block=16,
             N=256, short=False),
        # chunked prefill: 48 requests of up to 2048 new tokens in one 65536-token batch
        dict(name="slots_prefill", op="slots", B=48, most_added=2048, most_cached=16384, block=64,
             N=65536, short=False),
        # 16 sequences with their own sampling settings, logits as the BF16 head writes them
        dict(name="sample_mixed", op="sample", B=16, V=128256, dtype="bf16", policy="mixed"),
        # a rollout batch sampled from the whole distribution, binary32 logits
        dict(name="sample_rollout", op="sample", B=256, V=128256, dtype="fp32", policy="plain"),
    ]


def _log_int(rng, lo, hi):
    n = int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))
    n = min(max(n, lo), hi)
    return n + 1 if n == 3072 else n


def _kdim(rng):
    k = 128 * rng.randint(1, 64)
    return k + 128 if k == 3072 else k


def draw(rng):
    op = rng.choice(["norm", "norm_bwd", "rope", "rope_kv", "slots", "sample"])
    if op in ("norm", "norm_bwd"):
        K = _kdim(rng)
        M = _log_int(rng, 1, min(16384, (1 << 25) // K))
        if op == "norm":
            return dict(op=op, M=M, K=K, eps=rng.choice([1e-6, 1e-5]))
        return dict(op=op, M=M, K=K, n_dy=rng.randint(1, 3), dres=rng.random() < 0.7)
    if op in ("rope", "rope_kv"):
        D = rng.choice([64, 80, 96, 128, 192, 256])
        Hk = rng.choice([1, 2, 4, 8])
        Hq = Hk * rng.choice([1, 4, 8])
        T = _log_int(rng, 1, min(16384, (1 << 26) // ((Hq + Hk) * D)))
        R = rng.choice([D, D, D // 2, D // 4 + 2])
        c = dict(op=op, T=T, Hq=Hq, Hk=Hk, D=D, R=R - R % 2,
                 layout=rng.choice(["half", "interleaved"]),
                 scaling=rng.choice(["none", "linear", "wavelength"]),
                 factor=rng.choice([2.0, 4.0, 8.0]), packed=rng.random() < 0.5,
                 start=_log_int(rng, 1, 1 << 20))
        if op == "rope":
            return dict(c, backward=rng.random() < 0.5)
        return dict(c, S=T + _log_int(rng, 1, 16384))
    if op == "slots":
        B = _log_int(rng, 1, 1024)
        add = rng.choice([1, 1, _log_int(rng, 2, 65536 // B if B < 32768 else 2)])
        return dict(op=op, B=B, most_added=add, most_cached=_log_int(rng, 1, 16384),
                    block=rng.choice([8, 16, 32, 64, 24]), N=B * add, short=rng.random() < 0.2)
    V = rng.choice([32000, 50257, 128256, 151937, _log_int(rng, 100, 150000)])
    return dict(op=op, B=_log_int(rng, 1, min(256, (1 << 24) // V)), V=V,
                dtype=rng.choice(["bf16", "fp32"]),
                policy=rng.choice(["plain", "topk", "nucleus", "mixed"]))


# --------------------------------------------------------------------------
# what a user's program has in hand
# --------------------------------------------------------------------------

def _gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(int(seed))
    return g


def _randn(shape, g, std=1.0, dtype=BF16):
    return (torch.randn(shape, generator=g, device=DEV) * std).to(dtype)


def _empty(shape, dtype):
    return torch.empty(shape, dtype=dtype, device=DEV)


def _frequencies(case):
    """Angle per position of each pair (binary64): base^(-2i/R), scaled for long contexts."""
    base, R = 500000.0, case["R"]
    f = base ** (-torch.arange(0, R, 2, dtype=F64) / R)
    if case["scaling"] == "linear":
        f = f / case["factor"]
    elif case["scaling"] == "wavelength":
        turns = 8192.0 * f / (2 * math.pi)  # turns over the original context
        s = ((turns - 1.0) / (4.0 - 1.0)).clamp(0.0, 1.0)
        f = f * ((1 - s) / case["factor"] + s)
    return f.to(DEV)


def _heads(case, g, n_k):
    """q and n_k tensors of Hk heads: [T, H, D] views of one projection's rows, or separate."""
    T, D = case["T"], case["D"]
    counts = [case["Hq"]] + [case["Hk"]] * n_k
    if not case["packed"]:
        return [_randn((T, h, D), g) for h in counts]
    rows = _randn((T, sum(counts) * D), g)
    at, out = 0, []
    for h in counts:
        out.append(rows[:, at:at + h * D].unflatten(1, (h, D)))
        at += h * D
    return out


def prepare(case, seed):
    g, op = _gen(seed), case["op"]
    s = dict(case=dict(case))
    if op == "norm":
        M, K = case["M"], case["K"]
        x = torch.randn((M, K), generator=g, device=DEV)
        x[:, torch.randperm(K, generator=g, device=DEV)[:max(1, K // 1000)]] *= 50.0
        s |= dict(x=x.to(BF16), d=_randn((M, K), g, 0.5),
                  g=(1 + 0.1 * torch.randn((K,), generator=g, device=DEV)).to(BF16),
                  h=_empty((M, K), BF16), q=_empty((M, K), U8), s=_empty((K // 128, M), F32),
                  rstd=_empty((M,), F32))
    elif op == "norm_bwd":
        M, K = case["M"], case["K"]
        h = _randn((M, K), g)
        s |= dict(h=h, rstd=torch.rsqrt(h.double().square().mean(1) + 1e-5).float(),
                  g=(1 + 0.1 * torch.randn((K,), generator=g, device=DEV)).to(BF16),
                  dys=[_randn((M, K), g, 1e-3) for _ in range(case["n_dy"])],
                  dres=_randn((M, K), g, 1e-3) if case["dres"] else None,
                  dx=_empty((M, K), BF16), dg=_empty((K,), F32))
    elif op == "rope":
        q, k = _heads(case, g, 1)
        start = case["start"]
        s |= dict(q=q, k=k, freq=_frequencies(case),
                  pos=torch.arange(start, start + case["T"], device=DEV),
                  qo=_empty(q.shape, BF16), ko=_empty(k.shape, BF16))
    elif op == "rope_kv":
        q, k, v = _heads(case, g, 2)
        T, H, D, S = case["T"], case["Hk"], case["D"], case["S"]
        s |= dict(q=q, k=k, v=v, freq=_frequencies(case),
                  pos=torch.randint(0, case["start"] + 1, (T,), generator=g, device=DEV)
                  + torch.arange(T, device=DEV),
                  slots=torch.randperm(S, generator=g, device=DEV)[:T],
                  ks=torch.rand((H,), generator=g, device=DEV) * 0.01 + 0.008,
                  vs=torch.rand((H,), generator=g, device=DEV) * 0.01 + 0.008,
                  qo=_empty(q.shape, BF16),
                  kc=torch.zeros((S, H, D), dtype=U8, device=DEV),
                  vc=torch.zeros((S, H, D), dtype=U8, device=DEV))
    elif op == "slots":
        B, N, bs = case["B"], case["N"], case["block"]
        cached = torch.randint(0, case["most_cached"] + 1, (B,), generator=g, device=DEV)
        added = torch.randint(1 if case["most_added"] == 1 else 0, case["most_added"] + 1, (B,),
                              generator=g, device=DEV)
        width = (case["most_cached"] + case["most_added"] + bs - 1) // bs
        old = (cached + bs - 1) // bs
        new = (cached + added + bs - 1) // bs
        held, need = int(old.sum()), int((new - old).sum())
        ids = torch.randperm(held + need + 64, generator=g, device=DEV).to(I32)
        j = torch.arange(width, device=DEV)
        at = torch.cumsum(old, 0)[:, None] - old[:, None] + j
        table = torch.where(j < old[:, None], ids[at.clamp(max=held + need)], -1).to(I32)
        free = ids[held:held + (need // 2 if case["short"] else need + 64)].contiguous()
        s |= dict(cached=cached.to(I32), added=added.to(I32), table=table, free=free,
                  next=torch.zeros((1,), dtype=I64, device=DEV), offsets=_empty((B + 1,), I64),
                  pos=_empty((N,), I64), slots=_empty((N,), I64), rows=_empty((N,), I32),
                  counts=_empty((2,), I64))
    else:
        B, V = case["B"], case["V"]
        ld = (V + 7) // 8 * 8 if V % 2 == 0 else V
        x = torch.randn((B, ld), generator=g, device=DEV) * 2.5
        peaks = torch.randint(0, V, (B, 48), generator=g, device=DEV)
        x.scatter_add_(1, peaks, 3 + 4 * torch.rand((B, 48), generator=g, device=DEV))
        x[:, torch.randint(0, V, (max(1, V // 1000),), generator=g, device=DEV)] = NEG
        s |= dict(x=x.to(F32 if case["dtype"] == "fp32" else BF16)[:, :V],
                  u=torch.rand((B,), generator=g, device=DEV), T=None, k=None, p=None, m=None,
                  token=_empty((B,), I64), logp=_empty((B,), F32), logp_all=_empty((B,), F32),
                  kept=_empty((B,), I32))
        r = torch.arange(B, device=DEV)
        f = lambda vals, n, t: torch.tensor(vals, device=DEV, dtype=t)[(r // n) % len(vals)]
        if case["policy"] in ("topk", "mixed"):
            s["T"] = f([0.6, 1.0, 1.3], 1, F32)
            s["k"] = f([50, 20, 1000], 1, I32)
        if case["policy"] in ("nucleus", "mixed"):
            s["T"] = f([1.0, 0.7], 1, F32)
            s["p"] = f([0.95, 0.9, 0.5], 1, F32)
        if case["policy"] == "mixed":
            s["T"] = f([1.0, 0.6, 0.0, 1.3], 1, F32)
            s["k"] = f([0, 50, 0, 1000, 7], 1, I32)
            s["p"] = f([0.95, 1.0, 0.9], 2, F32)
            s["m"] = f([0.0, 0.05], 3, F32)
    return s


# --------------------------------------------------------------------------
# one pass
# --------------------------------------------------------------------------

def run(s):
    return (_own if own else _plain)(s)


def _own(s):
    import fp8_block_quantized_gb300 as jet
    c = s["case"]
    op = c["op"]
    if op == "norm":
        jet.jet_add_rmsnorm_quant_1x128(s["x"], s["d"], s["g"], c["eps"], s["h"], s["q"], s["s"],
                                        s["rstd"])
        return dict(h=s["h"], q=s["q"].view(F8), s=s["s"], rstd=s["rstd"])
    if op == "norm_bwd":
        jet.jet_add_rmsnorm_bwd(s["h"], s["g"], s["rstd"], s["dys"], s["dres"], s["dx"], s["dg"])
        return dict(dx=s["dx"], dg=s["dg"])
    if op == "rope":
        jet.jet_rope(s["q"], s["k"], s["freq"], s["pos"], s["qo"], s["ko"], c["layout"],
                     mscale=1.0, backward=c["backward"])
        return dict(q=s["qo"], k=s["ko"])
    if op == "rope_kv":
        jet.jet_rope_kv_cache_write(s["q"], s["k"], s["v"], s["freq"], s["pos"], s["ks"], s["vs"],
                                    s["slots"], s["qo"], s["kc"], s["vc"], c["layout"], mscale=1.0)
        return dict(q=s["qo"], k=s["kc"].view(F8), v=s["vc"].view(F8))
    if op == "slots":
        jet.jet_kv_slot_map(s["cached"], s["added"], c["block"], s["table"], s["free"], s["next"],
                            s["offsets"], s["pos"], s["slots"], s["rows"], s["counts"])
        return {n: s[n] for n in ("table", "offsets", "pos", "slots", "rows", "counts")}
    jet.jet_sample(s["x"], s["u"], s["T"], s["k"], s["p"], s["m"], s["token"], s["logp"],
                   s["logp_all"], s["kept"])
    return {n: s[n] for n in ("token", "logp", "logp_all", "kept")}


def _plain(s):
    c = s["case"]
    return {"norm": _norm, "norm_bwd": _norm_bwd, "rope": _rope, "rope_kv": _rope_kv,
            "slots": _slots, "sample": _sample}[c["op"]](s, c)


def _norm(s, c):
    M, K = c["M"], c["K"]
    h = (s["x"].float() + s["d"].float()).to(BF16)
    v = h.float()
    rstd = 1.0 / torch.sqrt((v * v).sum(1) / K + c["eps"])
    y = (v * rstd[:, None] * s["g"].float()).view(M, K // 128, 128)
    amax = y.abs().amax(2)
    scale = torch.where(amax == 0, 1.0, amax / 448.0)
    q = (y / scale[:, :, None]).to(F8).view(M, K)
    return dict(h=h, q=q, s=scale.t().contiguous(), rstd=rstd)


def _norm_bwd(s, c):
    K = c["K"]
    xh = s["h"].float() * s["rstd"][:, None]
    dy = s["dys"][0].float()
    for t in s["dys"][1:]:
        dy = dy + t.float()
    u = dy * s["g"].float()
    dx = s["rstd"][:, None] * (u - xh * ((u * xh).sum(1, keepdim=True) / K))
    if s["dres"] is not None:
        dx = dx + s["dres"].float()
    return dict(dx=dx.to(BF16), dg=(dy * xh).sum(0))


def _rotate(x, cos, sin, layout):
    """Pairs of the first R channels of x [T, H, D] turned by the angles of cos, sin [T, R/2]."""
    R = 2 * cos.shape[1]
    cos, sin, x = cos[:, None], sin[:, None], x.float()
    if layout == "half":
        a, b = x[..., :R // 2], x[..., R // 2:R]
        y = torch.cat([a * cos - b * sin, b * cos + a * sin, x[..., R:]], -1)
    else:
        a, b = x[..., 0:R:2], x[..., 1:R:2]
        y = torch.stack([a * cos - b * sin, b * cos + a * sin], -1).flatten(-2)
        y = torch.cat([y, x[..., R:]], -1)
    return y.to(BF16)


def _angles(s):
    a = s["pos"].double()[:, None] * s["freq"]
    return torch.cos(a).float(), torch.sin(a).float()


def _rope(s, c):
    cos, sin = _angles(s)
    if c["backward"]:
        sin = -sin
    return dict(q=_rotate(s["q"], cos, sin, c["layout"]), k=_rotate(s["k"], cos, sin, c["layout"]))


def _rope_kv(s, c):
    cos, sin = _angles(s)
    q, k = (_rotate(s[n], cos, sin, c["layout"]) for n in ("q", "k"))
    for x, scale, cache in ((k, s["ks"], s["kc"]), (s["v"], s["vs"], s["vc"])):
        codes = (x.float() / scale[:, None]).clamp(-448.0, 448.0).to(F8)
        cache[s["slots"]] = codes.view(U8)
    return dict(q=q, k=s["kc"].view(F8), v=s["vc"].view(F8))


def _slots(s, c):
    bs, N = c["block"], c["N"]
    cached, added = s["cached"].long(), s["added"].long()
    width, F = s["table"].shape[1], s["free"].shape[0]
    offsets = torch.cat([added.new_zeros(1), torch.cumsum(added, 0)])
    old = (cached + bs - 1) // bs
    need = (((cached + added + bs - 1) // bs).clamp(max=width) - old).clamp(min=0)
    upto = torch.cumsum(need, 0)
    first = s["next"] + upto - need
    j = torch.arange(width, device=DEV)
    at = first[:, None] + j - old[:, None]
    fresh = (j >= old[:, None]) & (j < (old + need)[:, None])
    got = torch.where(at < F, s["free"][at.clamp(0, F - 1)], -1) if F else torch.full_like(at, -1)
    table = torch.where(fresh, got, s["table"]).to(I32)
    t = torch.arange(N, device=DEV)
    r = torch.searchsorted(offsets[1:], t, right=True)
    real = r < c["B"]
    row = r.clamp(max=c["B"] - 1)
    pos = cached[row] + t - offsets[row]
    block = pos // bs
    ids = torch.where(block < width, table[row, block.clamp(max=width - 1)].long(), -1)
    slots = torch.where(real & (ids >= 0), ids * bs + pos % bs, -1)
    end = torch.minimum(s["next"] + upto[-1], torch.full_like(s["next"], F))
    return dict(table=table, offsets=offsets, pos=torch.where(real, pos, 0), slots=slots,
                rows=torch.where(real, r, -1).to(I32),
                counts=torch.cat([end, s["next"] + upto[-1:] - end]))


def _sample(s, c):
    B, V = c["B"], c["V"]
    x = s["x"].float()
    x = torch.where(torch.isnan(x), NEG, x)
    T = s["T"] if s["T"] is not None else torch.ones((B,), device=DEV)
    k = s["k"] if s["k"] is not None else torch.zeros((B,), dtype=I32, device=DEV)
    k = torch.where(T > 0, torch.where(k > 0, k.long(), V), 1)
    rt = 1.0 / torch.where(T > 0, T, 1.0)
    d = x - x.amax(1, keepdim=True)
    w = torch.exp(torch.where(d == 0, 0.0, d * rt[:, None]))
    total = w.double().sum(1)
    keep = x > NEG
    if s["k"] is not None or s["p"] is not None or s["m"] is not None:
        xs, order = torch.sort(x, dim=1, descending=True, stable=True)
        ws = w.gather(1, order).double()
        ok = (torch.arange(V, device=DEV) < k[:, None]) & (xs > NEG)
        if s["p"] is not None:
            mass = torch.cumsum(ws * ok, 1)
            target = s["p"].double() * mass[:, -1]
            ok &= (mass - ws < target[:, None]) | (s["p"] >= 1)[:, None]
        if s["m"] is not None:
            ok &= ws >= s["m"].double()[:, None]
        keep = torch.zeros_like(ok).scatter(1, order, ok)
    cum = torch.cumsum(w.double() * keep, 1)
    S = cum[:, -1]
    token = (cum <= (s["u"].double() * S)[:, None]).sum(1)
    wt = w.gather(1, token[:, None])[:, 0].double()
    log = lambda all_: torch.where(2 * wt > all_, torch.log1p(-(all_ - wt) / all_),
                                   torch.log(wt / all_)).float()
    return dict(token=token, logp=log(S), logp_all=log(total), kept=keep.sum(1).to(I32))


# --------------------------------------------------------------------------
# the work a pass cannot do without
# --------------------------------------------------------------------------

def work(case):
    op = case["op"]
    if op == "norm":
        n = case["M"] * case["K"]
        return dict(bytes=n * (2 + 2 + 2 + 1 + 4 / 128) + 2 * case["K"] + 4 * case["M"], flops=8 * n)
    if op == "norm_bwd":
        n, nd = case["M"] * case["K"], case["n_dy"]
        return dict(bytes=n * (2 + 2 * nd + 2 * case["dres"] + 2) + 6 * case["K"] + 4 * case["M"],
                    flops=(9 + nd) * n)
    if op == "rope":
        n = case["T"] * (case["Hq"] + case["Hk"]) * case["D"]
        return dict(bytes=4 * n + 8 * case["T"] + 4 * case["R"], flops=3 * n)
    if op == "rope_kv":
        nq, nk = (case["T"] * case[h] * case["D"] for h in ("Hq", "Hk"))
        return dict(bytes=4 * nq + 2 * 3 * nk + 16 * case["T"] + 4 * case["R"],
                    flops=3 * (nq + nk) + 2 * nk)
    if op == "slots":
        B, N = case["B"], case["N"]
        return dict(bytes=16 * B + 20 * N + 8 * ((N + case["block"] - 1) // case["block"]),
                    flops=8 * N)
    n = case["B"] * case["V"]
    return dict(bytes=n * (4 if case["dtype"] == "fp32" else 2) + 28 * case["B"], flops=4 * n)


# --------------------------------------------------------------------------
# the same in 64 bits
# --------------------------------------------------------------------------

def exact(case, seed):
    s, op = prepare(case, seed), case["op"]
    if op == "norm":
        h = s["x"].double().add_(s["d"])
        v = h.to(BF16).double()  # the stream holds BF16, and the norm is of what it holds
        rstd = (v.square().mean(1) + case["eps"]).rsqrt()
        y = torch.einsum("mk,m,k->mk", v, rstd, s["g"].double()).unflatten(1, (-1, 128))
        top = y.abs().amax(2) / 448
        scale = top + (top == 0)
        return dict(h=h, q=(y / scale[..., None]).flatten(1), s=scale.t(), rstd=rstd)
    if op == "norm_bwd":
        h, r, g = s["h"].double(), s["rstd"].double()[:, None], s["g"].double()
        dy = sum(t.double() for t in s["dys"])
        along = torch.einsum("mk,mk,k->m", dy, h, g)[:, None]
        dx = r * g * dy - h * r ** 3 * along / case["K"]
        if case["dres"]:
            dx += s["dres"].double()
        return dict(dx=dx, dg=torch.einsum("mk,mk,m->k", dy, h, r[:, 0]))
    if op in ("rope", "rope_kv"):
        angle = torch.outer(s["pos"].double(), s["freq"])
        turn = torch.polar(torch.ones_like(angle), -angle if case.get("backward") else angle)[:, None]
        half, R = case["layout"] == "half", case["R"]

        def rot(x):
            x = x.double()
            a, b = (x[..., :R // 2], x[..., R // 2:R]) if half else (x[..., :R:2], x[..., 1:R:2])
            z = torch.view_as_real(torch.complex(a, b) * turn)
            z = z.transpose(-1, -2).flatten(-2) if half else z.flatten(-2)
            return torch.cat([z, x[..., R:]], -1)
        q, k = rot(s["q"]), rot(s["k"])
        if op == "rope":
            return dict(q=q, k=k)

        def cached(x, scale):
            out = torch.zeros((case["S"],) + tuple(x.shape[1:]), dtype=F64, device=DEV)
            out[s["slots"]] = (x / scale.double()[None, :, None]).clamp(-448, 448)
            return out
        return dict(q=q, k=cached(k, s["ks"]), v=cached(s["v"].double(), s["vs"]))
    if op == "slots":
        return None
    # weights from binary32 differences and quotients, as the definition says; all else in 64 bits
    x = s["x"].float().nan_to_num(nan=NEG, posinf=math.inf, neginf=NEG)
    out = dict(token=None, logp=[], logp_all=[], kept=None)
    for b in range(case["B"]):
        T = float(s["T"][b]) if s["T"] is not None else 1.0
        k = int(s["k"][b]) if s["k"] is not None else 0
        k = 1 if T <= 0 else k if k > 0 else case["V"]
        inv = 1.0 / torch.tensor(T if T > 0 else 1.0, device=DEV)
        w = ((x[b] - x[b].max()) * inv).double().exp()
        full = w.sum()
        p = float(s["p"][b]) if s["p"] is not None else 1.0
        by = torch.argsort(x[b], descending=True, stable=True)[:k]
        if p < 1:
            run_ = w[by].cumsum(0)
            by = by[:1 + int((run_ < p * run_[-1]).sum())]
        if s["m"] is not None:
            by = by[w[by] >= float(s["m"][b])]
        by = by[x[b][by] > NEG].sort().values
        run_ = w[by].cumsum(0)
        at = by[torch.searchsorted(run_, s["u"][b].double() * run_[-1], right=True)]
        for name, everything in (("logp", run_[-1]), ("logp_all", full)):
            out[name].append((w[at] / everything).log())
    return dict(out, logp=torch.stack(out["logp"]), logp_all=torch.stack(out["logp_all"]))
