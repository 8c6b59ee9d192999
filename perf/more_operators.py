"""What a reinforcement-learning step needs between the FP8 cache and the weights'
gradients: what is measured, and their plain forms.

Attention over the paged FP8 KV cache (decoding, chunks of a prompt, and groups
of requests that share a prefix), the log-probabilities of given tokens under
the head without its logits, their gradient, and the gated activation's backward
with the 1x128 quantization.  ``run`` computes them with elementary torch
operations where ``own`` is false, and calls the package's entry points where it
is true.  ``exact`` is the same definition in 64 bits, written apart.
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
        # one user's chat: a single request decoding at a few thousand tokens
        dict(name="attn_decode_one", op="attn", B=1, new=1, least=4001, most=4001, group=0, prefix=0,
             Hq=32, Hk=8, D=128, block=16),
        # a decoding step of 64 requests of mixed lengths, the 8B-shaped model's heads
        dict(name="attn_decode", op="attn", B=64, new=1, least=17, most=8192, group=0, prefix=0,
             Hq=32, Hk=8, D=128, block=16),
        # two requests decoding far into a long context, the 32B-shaped model's heads
        dict(name="attn_decode_long", op="attn", B=2, new=1, least=100003, most=131072, group=0,
             prefix=0, Hq=64, Hk=8, D=128, block=64),
        # a rollout step: 16 prompts, 16 responses of each, a prompt's keys read once for all of them
        dict(name="attn_group", op="attn", B=256, new=1, least=1, most=1024, group=16, prefix=8192,
             Hq=32, Hk=8, D=128, block=16),
        # one long prompt shared by 128 responses, the 32B-shaped model's heads
        dict(name="attn_group_long", op="attn", B=128, new=1, least=64, most=256, group=128,
             prefix=32768, Hq=64, Hk=8, D=128, block=64),
        # chunked prefill: eight requests of up to 1024 new tokens behind cached ones
        dict(name="attn_prefill", op="attn", B=8, new=1024, least=1024, most=4096, group=0, prefix=0,
             Hq=32, Hk=8, D=128, block=64),
        # scoring a few tokens of a small model
        dict(name="head_small", op="head", T=48, K=512, V=2048, temperature=1.0, ignored=0.0),
        # the training forward's log-probabilities of the 8B-shaped model, 4096 tokens
        dict(name="head_train8b", op="head", T=4096, K=4096, V=128256, temperature=1.0, ignored=0.0),
        # their gradient: of the hidden states and of the head
        dict(name="head_bwd_train8b", op="head_bwd", T=4096, K=4096, V=128256, temperature=1.0,
             ignored=0.0),
        # a ragged batch with its prompts' tokens ignored, an odd vocabulary, sampled at 0.7
        dict(name="head_bwd_ragged", op="head_bwd", T=1537, K=5120, V=50257, temperature=0.7,
             ignored=0.3),
        # the gated activation's backward of a small model, one group of tokens
        dict(name="swiglu_bwd_small", op="swiglu_bwd", M=128, F=1024, joined=False),
        # the same in a training step of the 8B-shaped layer, gate and up from one product
        dict(name="swiglu_bwd_train8b", op="swiglu_bwd", M=8192, F=14336, joined=True),
    ]


def _log_int(rng, lo, hi):
    return min(max(int(round(math.exp(rng.uniform(math.log(lo), math.log(hi))))), lo), hi)


def draw(rng):
    op = rng.choice(["attn", "attn", "attn", "head", "head_bwd", "swiglu_bwd"])
    if op == "attn":
        D, Hk = rng.choice([64, 128, 128, 256]), rng.choice([1, 2, 4, 8])
        Hq = Hk * rng.choice([1, 3, 4, 8])
        kind = rng.choice(["decode", "group", "chunk"])
        c = dict(op=op, Hq=Hq, Hk=Hk, D=D, block=rng.choice([8, 16, 24, 64, 128]), group=0, prefix=0)
        room = (1 << 28) // (Hk * D)       # keys of all requests
        if kind == "decode":
            B = _log_int(rng, 1, 256)
            most = _log_int(rng, 1, min(131072, room // B))
            return dict(c, B=B, new=rng.choice([1, 1, 2, 5]), least=max(1, most // 8), most=most)
        if kind == "group":
            group = _log_int(rng, 2, 64)
            B = group * _log_int(rng, 1, 128 // group)
            most = _log_int(rng, 1, min(2048, room // B // 2))
            prefix = _log_int(rng, 1, min(32768, room // B // 2))
            return dict(c, B=B, new=1, least=1, most=most, group=group, prefix=prefix)
        B = _log_int(rng, 1, 16)
        new = _log_int(rng, 3, 8192 // B)
        most = new + _log_int(rng, 1, min(8192, (1 << 30) // (B * new * Hq)))
        return dict(c, B=B, new=new, least=new, most=most)
    if op in ("head", "head_bwd"):
        K = 8 * _log_int(rng, 8, 640)
        V = rng.choice([32000, 50257, 128256, 151937, _log_int(rng, 100, 150000)])
        T = _log_int(rng, 1, min(8192, (1 << 39) // (K * V)))
        return dict(op=op, T=T, K=K, V=V, temperature=rng.choice([1.0, 1.0, 0.7, 1.3]),
                    ignored=rng.choice([0.0, 0.3]))
    F = 128 * _log_int(rng, 1, 200)
    M = 128 * _log_int(rng, 1, min(64, (1 << 26) // (128 * F)))
    return dict(op=op, M=M, F=F, joined=rng.random() < 0.5)


def _lengths(case):
    """(new tokens, total length) of each request and the prefix of each group: ragged, by the case alone."""
    B, n = case["B"], case["new"]
    part = lambda b, r: (b * r + 0.5) % 1.0
    new = [n if n <= 2 else 1 + int(part(b, 0.7548776662) * n) for b in range(B)]
    own_ = [case["least"] + int(part(b, 0.6180339887) * (case["most"] - case["least"] + 1))
            for b in range(B)]
    if not case["group"]:
        return new, [max(a, m) for a, m in zip(own_, new)], []
    prefix = [case["prefix"] - int(part(i, 0.4142135624) * (case["prefix"] // 2))
              for i in range(B // case["group"])]
    return new, [prefix[b // case["group"]] + max(a, m) for b, (a, m) in enumerate(zip(own_, new))], prefix


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


def _codes(shape, g):
    """E4M3 codes of normal entries whose largest is about the format's."""
    return _randn(shape, g, 90.0, F32).clamp_(-448.0, 448.0).to(F8).view(U8)


def prepare(case, seed):
    g, op = _gen(seed), case["op"]
    s = dict(case=dict(case))
    if op == "attn":
        B, Hq, Hk, D, bs, per = (case[n] for n in ("B", "Hq", "Hk", "D", "block", "group"))
        new, total, prefix = _lengths(case)
        width = (max(total) + bs - 1) // bs
        need = torch.tensor([(t + bs - 1) // bs for t in total], device=DEV)
        j = torch.arange(width, device=DEV)
        lead = torch.arange(B, device=DEV)
        shared = torch.zeros((B,), dtype=I64, device=DEV)
        if per:                            # whole blocks of the prefix are the first request's
            lead = lead // per * per
            shared = torch.tensor(prefix, device=DEV)[torch.arange(B, device=DEV) // per] // bs
        first = torch.arange(B, device=DEV) == lead
        mine = (j < need[:, None]) & ((j >= shared[:, None]) | first[:, None])
        blocks = int(mine.sum())
        ids = torch.randperm(blocks, generator=g, device=DEV)
        at = (torch.cumsum(mine.flatten(), 0) - 1).view(B, width)
        table = torch.where(mine, ids[at.clamp(min=0)], -1)
        table = torch.where((j < shared[:, None]) & ~first[:, None], table[lead], table)
        T = sum(new)
        rows = _randn((T, (Hq + 2 * Hk) * D), g, 1.5)      # q among k and v of one projection
        s |= dict(q=rows[:, :Hq * D].unflatten(1, (Hq, D)),
                  k=_codes((blocks * bs, Hk, D), g), v=_codes((blocks * bs, Hk, D), g),
                  ks=torch.rand((Hk,), generator=g, device=DEV) * 0.005 + 0.008,
                  vs=torch.rand((Hk,), generator=g, device=DEV) * 0.005 + 0.008,
                  table=table.to(I32), offsets=torch.tensor([0] + new, device=DEV).cumsum(0),
                  lengths=torch.tensor(total, dtype=I32, device=DEV), longest=max(total),
                  newest=max(new), po=None, pl=None,
                  out=_empty((T, Hq, D), BF16), lse=_empty((T, Hq), F32))
        if per:
            s |= dict(po=torch.arange(0, B + 1, per, device=DEV),
                      pl=torch.tensor(prefix, dtype=I32, device=DEV))
    elif op in ("head", "head_bwd"):
        T, K, V = case["T"], case["K"], case["V"]
        w = _randn((V, K), g, 2.5 * K ** -0.5)
        target = torch.randint(0, V, (T,), generator=g, device=DEV)
        x = torch.randn((T, K), generator=g, device=DEV)
        x += w[target].float() * torch.rand((T, 1), generator=g, device=DEV) * 1.5
        if case["ignored"]:
            target[torch.rand((T,), generator=g, device=DEV) < case["ignored"]] = -100
        s |= dict(x=x.to(BF16), w=w, target=target, scale=1.0 / case["temperature"],
                  logp=_empty((T,), F32), lse=_empty((T,), F32))
        if op == "head_bwd":
            z = s["x"] @ w.t()             # stands in for the forward's result
            s |= dict(lse=torch.logsumexp(z.float() * s["scale"], 1), dlogp=_randn((T,), g, 1.0 / T, F32),
                      dx=_empty((T, K), BF16), dw=_empty((V, K), BF16))
    else:
        M, F = case["M"], case["F"]
        if case["joined"]:
            rows = _randn((M, 2 * F), g)
            gate, up = rows[:, :F], rows[:, F:]
        else:
            gate, up = _randn((M, F), g), _randn((M, F), g)
        s |= dict(gate=gate, up=up, dh=_randn((M, F), g, 1e-3),
                  qg=_empty((M, F), U8), sg=_empty((F // 128, M), F32),
                  qu=_empty((M, F), U8), su=_empty((F // 128, M), F32))
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
    if op == "attn":
        jet.jet_kv_attention(s["q"], s["k"], s["v"], s["ks"], s["vs"], s["table"], c["block"],
                             s["offsets"], s["lengths"], s["out"], s["lse"], s["po"], s["pl"])
        return dict(out=s["out"], lse=s["lse"])
    if op == "head":
        jet.jet_head_logp(s["x"], s["w"], s["target"], s["scale"], s["logp"], s["lse"])
        return dict(logp=s["logp"], lse=s["lse"])
    if op == "head_bwd":
        jet.jet_head_logp_bwd(s["x"], s["w"], s["target"], s["lse"], s["dlogp"], s["scale"], s["dx"],
                              s["dw"])
        return dict(dx=s["dx"], dw=s["dw"])
    jet.jet_swiglu_bwd_quant_1x128(s["gate"], s["up"], s["dh"], s["qg"], s["sg"], s["qu"], s["su"])
    return dict(qg=s["qg"].view(F8), sg=s["sg"], qu=s["qu"].view(F8), su=s["su"])


def _plain(s):
    c = s["case"]
    return {"attn": _attn, "head": _head, "head_bwd": _head_bwd, "swiglu_bwd": _swiglu_bwd}[c["op"]](s, c)


def _attn(s, c):
    B, Hq, Hk, D, bs = (c[n] for n in ("B", "Hq", "Hk", "D", "block"))
    T, L, n = s["q"].shape[0], s["longest"], s["newest"]
    off, length = s["offsets"], s["lengths"].long()
    new = off[1:] - off[:-1]
    b, p = torch.arange(B, device=DEV), torch.arange(L, device=DEV)
    reads = b[:, None].expand(B, L)
    if s["po"] is not None:
        i = torch.searchsorted(s["po"][1:], b, right=True)
        reads = torch.where(p < s["pl"][i].long()[:, None], s["po"][i][:, None], reads)
    slot = s["table"].long()[reads, p // bs] * bs + p % bs                       # [B, L]
    seen = p < length[:, None]
    slot = torch.where(seen, slot, 0)
    token = torch.searchsorted(off[1:], torch.arange(T, device=DEV), right=True)
    j = torch.arange(T, device=DEV) - off[token]
    q = torch.zeros((B, n, Hq, D), device=DEV)
    q[token, j] = s["q"].float()
    q = q.view(B, n, Hk, Hq // Hk, D).permute(0, 2, 3, 1, 4).reshape(B, Hk, Hq // Hk * n, D)
    k = s["k"].view(F8)[slot].float().mul_(s["ks"][:, None]).transpose(1, 2)     # [B, Hk, L, D]
    x = torch.matmul(q, k.transpose(2, 3)).mul_(D ** -0.5).view(B, Hk, Hq // Hk, n, L)
    del k
    pos = length[:, None] - new[:, None] + torch.arange(n, device=DEV)           # [B, n]
    x.masked_fill_((p > pos[..., None])[:, None, None], NEG)
    top = x.amax(-1, keepdim=True)
    x.sub_(torch.where(top > NEG, top, 0.0)).exp_()
    total = x.sum(-1, keepdim=True)
    v = s["v"].view(F8)[slot].float().mul_(s["vs"][:, None]).transpose(1, 2)
    o = torch.matmul(x.view(B, Hk, -1, L), v).view(B, Hk, Hq // Hk, n, D) / total
    o = o.permute(0, 3, 1, 2, 4).reshape(B, n, Hq, D)
    lse = (top + torch.log(total))[..., 0].permute(0, 3, 1, 2).reshape(B, n, Hq)
    return dict(out=o[token, j].to(BF16), lse=lse[token, j])


def _head(s, c):
    z = (s["x"].float() @ s["w"].float().t()).mul_(s["scale"])
    top = z.amax(1)
    t = s["target"]
    ok = (t >= 0) & (t < c["V"])
    at = z.gather(1, torch.where(ok, t, 0)[:, None])[:, 0]
    lse = top + torch.log(z.sub_(top[:, None]).exp_().sum(1))
    return dict(logp=torch.where(ok, at - lse, 0.0), lse=lse)


def _head_bwd(s, c):
    x, w, t = s["x"].float(), s["w"].float(), s["target"]
    ok = (t >= 0) & (t < c["V"])
    z = (x @ w.t()).mul_(s["scale"])
    d = z.sub_(s["lse"][:, None]).exp_().neg_()
    d.scatter_add_(1, torch.where(ok, t, 0)[:, None], torch.ones_like(t, dtype=F32)[:, None])
    d.mul_(torch.where(ok, s["dlogp"] * s["scale"], 0.0)[:, None])
    return dict(dx=(d @ w).to(BF16), dw=(d.t() @ x).to(BF16))


def _swiglu_bwd(s, c):
    M, F = c["M"], c["F"]
    gate, up, dh = s["gate"].float(), s["up"].float(), s["dh"].float()
    sig = 1.0 / (1.0 + torch.exp(-gate))
    dup = dh * (gate * sig)
    dgate = dh * up * (sig * (1.0 + gate * (1.0 - sig)))

    def quant(y):
        y = y.view(M, F // 128, 128)
        amax = y.abs().amax(2)
        scale = torch.where(amax == 0, 1.0, amax / 448.0)
        return (y / scale[:, :, None]).to(F8).view(M, F), scale.t().contiguous()
    qg, sg = quant(dgate)
    qu, su = quant(dup)
    return dict(qg=qg, sg=sg, qu=qu, su=su)


# --------------------------------------------------------------------------
# the work a pass cannot do without
# --------------------------------------------------------------------------

def work(case):
    op = case["op"]
    if op == "attn":
        Hq, Hk, D, per = case["Hq"], case["Hk"], case["D"], case["group"]
        new, total, prefix = _lengths(case)
        keys = sum(total) - sum(p * (per - 1) for p in prefix)      # a shared prefix once
        pairs = sum(n * t - n * (n - 1) // 2 for n, t in zip(new, total))
        T = sum(new)
        blocks = sum((t + case["block"] - 1) // case["block"] for t in total)
        return dict(bytes=2 * keys * Hk * D + 4 * T * Hq * D + 4 * T * Hq + 4 * blocks + 8 * Hk
                    + 12 * case["B"], flops=4 * pairs * Hq * D)
    if op in ("head", "head_bwd"):
        T, K, V = case["T"], case["K"], case["V"]
        if op == "head":
            return dict(bytes=2 * K * (T + V) + 16 * T, flops=2 * T * K * V + 4 * T * V)
        kept = T - int(case["ignored"] * T)      # ignored rows have no gradient to compute
        return dict(bytes=4 * K * (T + V) + 16 * T, flops=6 * kept * K * V + 5 * kept * V)
    n = case["M"] * case["F"]
    return dict(bytes=n * (3 * 2 + 2 * (1 + 4 / 128)), flops=20 * n)


# --------------------------------------------------------------------------
# the same in 64 bits
# --------------------------------------------------------------------------

def exact(case, seed):
    op = case["op"]
    if op in ("head", "head_bwd") and (2 if op == "head" else 6) * case["T"] * case["K"] * case["V"] > 1e13:
        return None
    s = prepare(case, seed)
    if op == "attn":
        Hq, Hk, D, bs = (case[n] for n in ("Hq", "Hk", "D", "block"))
        off, table, out, lses = s["offsets"].tolist(), s["table"].long(), [], []
        qd = s["q"].double() * D ** -0.5
        kd, vd = (lambda at: s["k"].view(F8)[at].double()), (lambda at: s["v"].view(F8)[at].double())
        for b, length in enumerate(s["lengths"].tolist()):
            at = torch.arange(length, device=DEV)
            row = torch.full_like(at, b)
            if case["group"]:
                i = b // case["group"]
                row[:int(s["pl"][i])] = int(s["po"][i])
            slots = bs * table[row, torch.div(at, bs, rounding_mode="floor")] + torch.remainder(at, bs)
            n = off[b + 1] - off[b]
            hidden = at[None] > length - n + torch.arange(n, device=DEV)[:, None]
            keys, values = kd(slots) * s["ks"].double()[None, :, None], vd(slots) * s["vs"].double()[None, :, None]
            queries = qd[off[b]:off[b + 1]].unflatten(1, (Hk, Hq // Hk))
            logits = torch.einsum("nhgd,lhd->hgnl", queries, keys).masked_fill(hidden, NEG)
            lse = torch.logsumexp(logits, -1)
            weights = torch.exp(logits - lse[..., None])
            out.append(torch.einsum("hgnl,lhd->nhgd", weights, values).flatten(1, 2))
            lses.append(lse.permute(2, 0, 1).flatten(1))
        return dict(out=torch.cat(out), lse=torch.cat(lses))
    if op in ("head", "head_bwd"):
        V, t = case["V"], s["target"]
        real = (t >= 0) & (t < V)
        logits = torch.mm(s["x"].double(), s["w"].double().t()) * float(s["scale"])
        if op == "head":
            lse = torch.logsumexp(logits, 1)
            chosen = logits[torch.arange(case["T"], device=DEV), t.clamp(0, V - 1)]
            return dict(logp=torch.where(real, chosen - lse, 0.0), lse=lse)
        probability = torch.exp(logits - s["lse"].double()[:, None])
        del logits
        up = torch.where(real, s["dlogp"].double(), 0.0) * float(s["scale"])
        rows = torch.nonzero(real)[:, 0]
        grad = probability.mul_(-up[:, None])
        grad[rows, t[rows]] += up[rows]
        return dict(dx=torch.mm(grad, s["w"].double()), dw=torch.mm(grad.t(), s["x"].double()))
    g, u, d = (s[n].double() for n in ("gate", "up", "dh"))
    gone = torch.sigmoid(-g)                        # 1 - sigmoid(g)
    parts = dict(g=d * u * (1 - gone) * (1 + g * gone), u=d * g * (1 - gone))
    out = {}
    for name, y in parts.items():
        y = y.unflatten(1, (-1, 128))
        top = y.abs().amax(2) / 448
        scale = top + (top == 0)
        out["q" + name], out["s" + name] = (y / scale[..., None]).flatten(1), scale.t()
    return {n: out[n] for n in ("qg", "sg", "qu", "su")}
