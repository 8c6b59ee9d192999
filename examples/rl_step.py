#!/usr/bin/env python3
"""One reinforcement-learning step of a small decoder in the unified FP8 flow:
a rollout over a paged FP8 KV cache, the training forward over the same
tokens, the mismatch metric between the two, and a backward through the last
layer.

    python examples/rl_step.py

The linear layers, the norms with their residual additions, the rotary
positions, the cache writes and slot maps, the rollout's attention over the cache,
the sampling, the drawn tokens' log-probabilities with their gradient, and the
gated activation's backward are the library's calls.  Embedding and the training
attention are plain torch, as they would be another library's in a real program.
"""
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import fp8_block_quantized_gb300 as jet  # noqa: E402

HIDDEN, HQ, HK, D, FFN, VOCAB, LAYERS, EPS = 512, 4, 2, 128, 1024, 2048, 2, 1e-5
BLOCK, BLOCKS, WIDTH = 16, 256, 8          # cache: 256 blocks of 16 slots, 8 blocks a request
BF16 = torch.bfloat16


class Model:
    """BF16 weights and, per weight sync, their FP8 form."""

    def __init__(self, seed=0, device="cuda"):
        g = torch.Generator().manual_seed(seed)
        w = lambda n, k: (torch.randn((n, k), generator=g) * k ** -0.5).to(BF16).to(device)
        gain = lambda: (1 + 0.1 * torch.randn((HIDDEN,), generator=g)).to(BF16).to(device)
        self.embed = (torch.randn((VOCAB, HIDDEN), generator=g)).to(BF16).to(device)
        self.layers = [dict(q=w(HQ * D, HIDDEN), k=w(HK * D, HIDDEN), v=w(HK * D, HIDDEN),
                            o=w(HIDDEN, HQ * D), gate=w(FFN, HIDDEN), up=w(FFN, HIDDEN),
                            down=w(HIDDEN, FFN), norm1=gain(), norm2=gain())
                       for _ in range(LAYERS)]
        self.head, self.norm = w(VOCAB, HIDDEN), gain()
        self.inv_freq, self.mscale = jet.rope_inv_freq(D, 10000.0, "wavelength", 4.0, 64.0, 1.0, 4.0,
                                                       device=device)
        self.sync()

    def sync(self):
        self.fp8 = [{n: jet.quant_w_128x128(t) for n, t in l.items() if t.dim() == 2}
                    for l in self.layers]
        self.fp8_head = jet.quant_w_128x128(self.head)

    def hidden(self, tokens, attend, save=None):
        """The 1x128 form of the tokens' hidden states behind the last norm;
        attend(layer, q, k, v) is the attention over [T, heads, D].  `save` (a dict)
        takes what the last layer's backward needs."""
        T = tokens.numel()
        x, d = self.embed[tokens], torch.zeros((T, HIDDEN), dtype=BF16, device=tokens.device)
        for i, (p, w) in enumerate(zip(self.layers, self.fp8)):
            x, n1, s1, r1 = jet.add_rmsnorm_quant_1x128(x, d, p["norm1"], EPS, with_rstd=True)
            q, k, v = (jet.gemm_fp8_fwd(n1, s1, *w[n]).unflatten(1, (-1, D)) for n in "qkv")
            a = attend(i, q, k, v)
            d = jet.gemm_fp8_fwd(*jet.quant_act_1x128(a), *w["o"])
            x2, n2, s2, r2 = jet.add_rmsnorm_quant_1x128(x, d, p["norm2"], EPS, with_rstd=True)
            gate, up = (jet.gemm_fp8_fwd(n2, s2, *w[n]) for n in ("gate", "up"))
            if save is not None:
                save.update(x1=x, r1=r1, x2=x2, r2=r2, gate=gate, up=up)
            d, x = jet.gemm_fp8_fwd(*jet.swiglu_quant_1x128(gate, up), *w["down"]), x2
        x, n, s, r = jet.add_rmsnorm_quant_1x128(x, d, self.norm, EPS, with_rstd=True)
        if save is not None:
            save.update(xf=x, rf=r)
        return n, s

    def logits(self, tokens, attend):
        return jet.gemm_fp8_fwd(*self.hidden(tokens, attend), *self.fp8_head)


def attention(q, k, v, q_pos, k_pos):
    """Causal grouped-query attention in binary32: q [T, HQ, D], k and v [L, HK, D]."""
    k, v = (t.float().repeat_interleave(HQ // HK, 1) for t in (k, v))
    s = torch.einsum("thd,lhd->htl", q.float(), k) * D ** -0.5
    s = s.masked_fill(k_pos[None, None] > q_pos[None, :, None], float("-inf"))
    return torch.einsum("htl,lhd->thd", torch.softmax(s, -1), v)


class PagedCache:
    """FP8 K and V of every layer in blocks shared by the requests."""

    def __init__(self, requests, device="cuda"):
        e = lambda: torch.zeros((BLOCKS * BLOCK, HK, D), dtype=torch.uint8, device=device)
        self.k, self.v = [e() for _ in range(LAYERS)], [e() for _ in range(LAYERS)]
        self.scale = [None] * LAYERS
        self.table = torch.full((requests, WIDTH), -1, dtype=torch.int32, device=device)
        self.free = torch.randperm(BLOCKS, device=device).to(torch.int32)
        self.next = torch.zeros((2,), dtype=torch.int64, device=device)
        self.length = torch.zeros((requests,), dtype=torch.int32, device=device)

    def step(self, model, tokens, added, capacity):
        """The model's logits of `added` new tokens a request, written to the cache."""
        offsets, pos, slots, rows, self.next = jet.kv_slot_map(
            self.length, added, BLOCK, self.table, self.free, self.next[:1], capacity)
        self.length += added

        def attend(i, q, k, v):
            if self.scale[i] is None:    # calibrated on the prompts after the weight sync
                self.scale[i] = (jet.kv_calibrate(jet.rope(k, None, model.inv_freq, pos,
                                                           mscale=model.mscale)[0]),
                                 jet.kv_calibrate(v.contiguous()))
            ks, vs = self.scale[i]
            qr = torch.empty_like(q)
            jet.jet_rope_kv_cache_write(q, k, v, model.inv_freq, pos, ks, vs, slots, qr, self.k[i],
                                        self.v[i], mscale=model.mscale)
            return jet.kv_attention(qr, self.k[i], self.v[i], ks, vs, self.table, BLOCK, offsets,
                                    self.length).flatten(1)

        return model.logits(tokens, attend), offsets


def rollout(model, prompts, steps, seed=1):
    """(sequences, logp of every drawn token [requests, steps]) sampled from the model."""
    dev = model.embed.device
    g = torch.Generator(device=dev).manual_seed(seed)
    B = len(prompts)
    cache = PagedCache(B, dev)
    settings = dict(temperature=torch.full((B,), 1.0, device=dev),
                    top_p=torch.full((B,), 0.95, device=dev))
    tokens = torch.cat(prompts)
    added = torch.tensor([p.numel() for p in prompts], dtype=torch.int32, device=dev)
    drawn, logps = [], []
    for _ in range(steps):
        logits, offsets = cache.step(model, tokens, added, tokens.numel())
        last = logits[offsets[1:] - 1].contiguous()
        u = torch.rand((B,), generator=g, device=dev)
        token, _, logp, _ = jet.sample(last, u, **settings)
        drawn.append(token)
        logps.append(logp)
        tokens, added = token, torch.ones_like(added)
    drawn = torch.stack(drawn, 1)
    return [torch.cat([p, d]) for p, d in zip(prompts, drawn)], torch.stack(logps, 1)


def train_forward(model, sequences, save=None):
    """Hidden states (BF16) of the concatenated sequences with BF16 keys and values,
    and the sequences' ranges."""
    ends = torch.tensor([s.numel() for s in sequences]).cumsum(0).tolist()
    ranges = list(zip([0] + ends[:-1], ends))
    pos = torch.cat([torch.arange(s.numel(), device=s.device) for s in sequences])

    def attend(i, q, k, v):
        qr, kr = jet.rope(q, k, model.inv_freq, pos, mscale=model.mscale)
        if save is not None:
            save.update(qr=qr, kr=kr, v=v, pos=pos, ranges=ranges)
        return torch.cat([attention(qr[a:b], kr[a:b], v[a:b], pos[a:b], pos[a:b])
                          for a, b in ranges]).flatten(1).to(BF16)

    codes, scales = model.hidden(torch.cat(sequences), attend, save)
    x = codes.view(torch.float8_e4m3fn).float() * scales.t().repeat_interleave(128, 1)
    return x.to(BF16), ranges


def backward_last_layer(model, save, dx):
    """Gradients of the last layer's norms and of its input from those of the
    hidden states: DGrads in FP8, the norms', the rotation's and the gated
    activation's backward, attention by autograd."""
    p, w = model.layers[-1], model.fp8[-1]

    def dgrad(dy, weight):
        return jet.gemm_fp8_dgrad(*jet.quant_act_1x128(dy.contiguous()), *weight)

    dx, dnorm = jet.add_rmsnorm_bwd(save["xf"], model.norm, save["rf"], [dx])
    qg, sg, qu, su = jet.swiglu_bwd_quant_1x128(save["gate"], save["up"], dgrad(dx, w["down"]))
    dx, dnorm2 = jet.add_rmsnorm_bwd(save["x2"], p["norm2"], save["r2"],
                                     [jet.gemm_fp8_dgrad(qg, sg, *w["gate"]),
                                      jet.gemm_fp8_dgrad(qu, su, *w["up"])], dx)
    da = dgrad(dx, w["o"]).float().unflatten(1, (HQ, D))
    q, k, v = (save[n].float().requires_grad_() for n in ("qr", "kr", "v"))
    a = torch.cat([attention(q[s:e], k[s:e], v[s:e], save["pos"][s:e], save["pos"][s:e])
                   for s, e in save["ranges"]])
    dq, dk, dv = (t.to(BF16) for t in torch.autograd.grad(a, (q, k, v), da))
    dq, dk = jet.rope(dq, dk, model.inv_freq, save["pos"], mscale=model.mscale, backward=True)
    dx, dnorm1 = jet.add_rmsnorm_bwd(save["x1"], p["norm1"], save["r1"],
                                     [dgrad(t.flatten(1), w[n]) for t, n in ((dq, "q"), (dk, "k"), (dv, "v"))],
                                     dx)
    return dict(norm=dnorm, norm2=dnorm2, norm1=dnorm1, x=dx)


def rl_step(requests=8, steps=24, seed=0):
    """One step; returns the metric, the loss and the last layer's gradients."""
    model = Model(seed)
    g = torch.Generator().manual_seed(seed + 1)
    prompts = [torch.randint(0, VOCAB, (int(n),), generator=g).cuda()
               for n in torch.randint(1, 40, (requests,), generator=g)]
    sequences, logp_rollout = rollout(model, prompts, steps, seed + 2)
    save = {}
    x, ranges = train_forward(model, sequences, save)
    # the drawn tokens' log-probabilities under the training forward: a token is the target
    # of the position before it, the prompts' are ignored
    target = torch.full((x.shape[0],), -100, device="cuda")
    at = torch.cat([torch.arange(e - steps - 1, e - 1) for _, e in ranges]).cuda()
    target[at] = torch.cat([s[-steps:] for s in sequences])
    logp, lse = jet.head_logp(x, model.head, target)
    logp_train = logp[at]
    metric, count, weight = jet.token_mismatch_masked(logp_train.contiguous(),
                                                      logp_rollout.flatten().contiguous(), cap=2.0)
    # policy gradient of -sum(weight * logp) with unit advantages
    dlogp = torch.zeros_like(logp)
    dlogp[at] = -weight / count
    dx, dhead = jet.head_logp_bwd(x, model.head, target, lse, dlogp)
    grads = backward_last_layer(model, save, dx)
    grads["head"] = dhead
    torch.cuda.synchronize()
    code, word = jet.device_status()
    assert code == 0, f"device status {code} ({word:#x})"
    return dict(metric=float(metric), loss=float(-(weight * logp_train).sum() / count), grads=grads,
                sequences=sequences, logp_rollout=logp_rollout, logp_train=logp_train)


if __name__ == "__main__":
    jet.load()
    r = rl_step()
    print(f"token-mult-prob-error {r['metric']:.4f}, loss {r['loss']:.4f}, gradient norms",
          {n: round(float(t.float().norm()), 4) for n, t in r["grads"].items()})
