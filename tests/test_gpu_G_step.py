"""GPU tests of the operators between the cache and the gradients as a step uses
them together: slots, rotary cache writes and attention over several steps; the
head's log-probabilities against the sampler's; the gated block's backward in FP8;
and calls from several threads at once."""
import threading

import pytest
import torch

pytestmark = pytest.mark.gpu
BF16, F8 = torch.bfloat16, torch.float8_e4m3fn
B, HQ, HK, D, BLOCK = 5, 8, 2, 128, 16


@pytest.fixture(scope="module")
def jet(torch_cuda):
    import fp8_block_quantized_gb300 as j
    j.load()
    return j


def test_a_cache_filled_in_steps(jet):
    """Prompts in two chunks, then single tokens: each step's attention equals that of
    the queries over all keys so far, as the cache holds them."""
    g = torch.Generator().manual_seed(1)
    dev = "cuda"
    freq, _ = jet.rope_inv_freq(D, 10000.0)
    ks = vs = torch.full((HK,), 0.012, device=dev)
    kc, vc = (torch.zeros((64 * BLOCK, HK, D), dtype=torch.uint8, device=dev) for _ in range(2))
    table = torch.full((B, 12), -1, dtype=torch.int32, device=dev)
    free = torch.randperm(64, generator=g).to(torch.int32).to(dev)
    nxt = torch.zeros((1,), dtype=torch.int64, device=dev)
    length = torch.zeros((B,), dtype=torch.int32, device=dev)
    seen = [([], []) for _ in range(B)]                    # rotated K and V of each request, from the cache
    for added in ([70, 3, 40, 100, 17], [30, 0, 41, 1, 60], [1] * 5, [1, 0, 1, 1, 0], [2, 1, 1, 5, 1]):
        add = torch.tensor(added, dtype=torch.int32, device=dev)
        cap = sum(added) + 3
        offsets, pos, slots, rows, counts = jet.kv_slot_map(length, add, BLOCK, table, free, nxt, cap)
        nxt = counts[:1].clone()
        length += add
        q, k, v = ((torch.randn((cap, h, D), generator=g)).to(BF16).to(dev) for h in (HQ, HK, HK))
        qr = torch.empty_like(q)
        jet.jet_rope_kv_cache_write(q, k, v, freq, pos, ks, vs, slots, qr, kc, vc)
        out, lse = jet.kv_attention(qr, kc, vc, ks, vs, table, BLOCK, offsets, length, with_lse=True)
        for b in range(B):
            lo, hi = offsets[b].item(), offsets[b + 1].item()
            for at in slots[lo:hi].tolist():
                seen[b][0].append(kc[at].view(F8).double() * ks.double()[:, None])
                seen[b][1].append(vc[at].view(F8).double() * vs.double()[:, None])
            n = hi - lo
            if n == 0:
                continue
            K, V = (torch.stack(s).repeat_interleave(HQ // HK, 1) for s in seen[b])
            x = torch.einsum("thd,lhd->htl", qr[lo:hi].double(), K) * D ** -0.5
            hidden = torch.arange(len(K), device=dev) > (len(K) - n + torch.arange(n, device=dev))[:, None]
            w = torch.softmax(x.masked_fill(hidden, float("-inf")), -1)
            ref = torch.einsum("htl,lhd->thd", w, V)
            mag = torch.einsum("htl,lhd->thd", w, V.abs())
            # BF16's half step, the weights' 2^-11 and the scores' rounding (|x| below 2^5)
            assert ((out[lo:hi].double() - ref).abs() <= 2.0 ** -8 * ref.abs() + 2.0 ** -10 * mag).all()
        assert not out[sum(added):].any() and (lse[sum(added):] == float("-inf")).all()


def test_the_head_agrees_with_the_sampler(jet):
    """Tokens drawn from the logits the head's product would write: their
    log-probabilities under all weights are the head's."""
    g = torch.Generator().manual_seed(2)
    T, K, V = 40, 256, 3001
    x = torch.randn((T, K), generator=g).to(BF16).cuda()
    w = (torch.randn((V, K), generator=g) * 2.5 * K ** -0.5).to(BF16).cuda()
    logits = x.float() @ w.float().t()
    u = torch.rand((T,), generator=g).cuda()
    temperature = torch.full((T,), 0.7, device="cuda")
    token, _, logp_all, _ = jet.sample(logits, u, temperature)
    logp, _ = jet.head_logp(x, w, token, 1 / 0.7)
    # binary32 logits of 256 products, twice (2^-20 of their size of 16 at most), weights to 2^-22
    assert ((logp - logp_all).abs() <= 2.0 ** -14).all()


def test_the_gated_block_backward(jet):
    """dx of the gated block from dh: the two DGrads of the quantized gradients
    against the formula on the dequantized operands."""
    g = torch.Generator().manual_seed(3)
    M, F, K = 192, 384, 256
    rnd = lambda *s: torch.randn(s, generator=g).to(BF16).cuda()
    gate, up, dh = rnd(M, F), rnd(M, F), rnd(M, F)
    wg, wu = (jet.quant_w_128x128((torch.randn((F, K), generator=g) * K ** -0.5).to(BF16).cuda()) for _ in range(2))
    qg, sg, qu, su = jet.swiglu_bwd_quant_1x128(gate, up, dh)
    got = jet.gemm_fp8_dgrad(qg, sg, *wg).double() + jet.gemm_fp8_dgrad(qu, su, *wu).double()
    G, U = gate.double(), up.double()
    s = torch.sigmoid(G)
    dg, du = dh.double() * U * s * (1 + G * (1 - s)), dh.double() * G * s
    W = [q.view(F8).double() * sc.double().repeat_interleave(128, 0).repeat_interleave(128, 1) for q, sc in (wg, wu)]
    ref = dg @ W[0] + du @ W[1]
    # each gradient is off by half an E4M3 step, 2^-4 of itself or of the group's smallest normal
    off = [2.0 ** -4 * d.abs() + 2.0 ** -10 * d.abs().view(M, -1, 128).amax(2).repeat_interleave(128, 1) / 448 for d in (dg, du)]
    bound = off[0] @ W[0].abs() + off[1] @ W[1].abs() + 2.0 ** -7 * (dg.abs() @ W[0].abs() + du.abs() @ W[1].abs())
    assert ((got - ref).abs() <= bound).all()
    assert (got - ref).norm() / ref.norm() < 2.0 ** -5


def test_threads_with_other_sizes(jet):
    """Several host threads, each with its own stream and sizes, give what each gives alone."""
    def attention(n, hq, d, long):
        g = torch.Generator().manual_seed(n)
        q = torch.randn((n, hq, d), generator=g).to(BF16).cuda()
        kc, vc = (torch.randn((n * long, 2, d), generator=g).mul(90).clamp(-448, 448).to(F8).view(torch.uint8).cuda()
                  for _ in range(2))
        sc = torch.full((2,), 0.01, device="cuda")
        table = torch.arange(n * (long // 16), dtype=torch.int32).view(n, -1).cuda()
        off = torch.arange(n + 1).cuda()
        length = torch.full((n,), long, dtype=torch.int32, device="cuda")
        return lambda s: jet.kv_attention(q, kc, vc, sc, sc, table, 16, off, length, stream=s)

    def head(T, K, V):
        g = torch.Generator().manual_seed(T)
        x, w = torch.randn((T, K), generator=g).to(BF16).cuda(), torch.randn((V, K), generator=g).mul(0.1).to(BF16).cuda()
        target, d = torch.randint(0, V, (T,), generator=g).cuda(), torch.randn((T,), generator=g).cuda()

        def call(s):
            logp, lse = jet.head_logp(x, w, target, stream=s)
            return torch.cat([t.flatten().float() for t in (logp, *jet.head_logp_bwd(x, w, target, lse, d, stream=s))])
        return call
    calls = [attention(3, 8, 128, 512), attention(40, 64, 64, 64), attention(7, 4, 256, 1024), head(20, 128, 999),
             head(300, 256, 2000)]
    torch.cuda.synchronize()
    want = [c(None) for c in calls]
    torch.cuda.synchronize()
    start, errors = threading.Barrier(len(calls)), []

    def work(call, ref):
        try:
            stream = torch.cuda.Stream()
            start.wait()
            for _ in range(40):
                got = call(stream)
            stream.synchronize()
            assert torch.equal(got, ref)
        except BaseException as e:  # noqa: BLE001  (told below, outside the thread)
            errors.append(e)
    threads = [threading.Thread(target=work, args=a) for a in zip(calls, want)]
    for th in threads:
        th.start()
    for th in threads:
        th.join()
    torch.cuda.synchronize()
    assert not errors, errors[0]
    code, word = jet.device_status()
    assert code == 0, hex(word)


def test_refusals(jet):
    e = lambda *s, d=BF16: torch.zeros(s, dtype=d, device="cuda")
    q, c, sc = e(2, 4, 128), e(32, 2, 128, d=torch.uint8), e(2, d=torch.float32)
    table, off, length = e(2, 1, d=torch.int32), torch.arange(3).cuda(), e(2, d=torch.int32)
    ok = dict(q=q, k_cache=c, v_cache=c, k_scale=sc, v_scale=sc, table=table, block_size=16, offsets=off,
              lengths=length)
    jet.kv_attention(**ok)
    for name, bad, error in (
            ("q", q[:, :, :64], ValueError), ("q", q.float(), TypeError), ("q", q.transpose(0, 1), ValueError),
            ("k_cache", c[:, :1], ValueError), ("v_cache", e(16, 2, 128, d=torch.uint8), ValueError),
            ("k_scale", e(1, d=torch.float32), ValueError), ("table", table.long(), TypeError),
            ("table", e(3, 1, d=torch.int32), ValueError), ("offsets", off[:2], ValueError),
            ("offsets", off.int(), TypeError), ("lengths", length.long(), TypeError),
            ("block_size", 0, jet.JetError), ("block_size", -16, jet.JetError)):
        with pytest.raises(error):
            jet.kv_attention(**dict(ok, **{name: bad}))
    for kw in (dict(scale=0.0), dict(scale=float("nan"))):
        with pytest.raises(jet.JetError):
            jet.kv_attention(**ok, **kw)
    with pytest.raises(ValueError):
        jet.kv_attention(**ok, prefix_offsets=torch.tensor([0, 2]).cuda())
    with pytest.raises(jet.JetError):                       # 3 query heads on 2 KV heads
        jet.kv_attention(**dict(ok, q=e(2, 3, 128)))
    with pytest.raises(jet.JetError):
        jet.jet_kv_attention(*ok.values(), torch.empty_like(q), ws=e(16, d=torch.uint8))
    with pytest.raises(ValueError):
        jet.swiglu_bwd_quant_1x128(e(4, 128), e(4, 256)[:, :128], e(4, 128))
    with pytest.raises(jet.JetError):
        jet.swiglu_bwd_quant_1x128(e(4, 100), e(4, 100), e(4, 100))
