"""GPU tests of the block tables and slot maps: every output against a plain
loop over the requests and their tokens."""
import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def jet(torch_cuda):
    import fp8_block_quantized_gb300 as j
    j.load()
    return j


def plain(cached, added, bs, table, free, nxt, N):
    table = table.copy()
    width, taken, lacking = table.shape[1], min(max(nxt, 0), len(free)), 0
    offsets, pos, slots, rows = [0], [], [], []
    for b, (c, n) in enumerate(zip(np.maximum(cached, 0).tolist(), np.maximum(added, 0).tolist())):
        for j in range(-(-c // bs), min(-(-(c + n) // bs), width)):
            if taken < len(free):
                table[b, j] = free[taken]
                taken += 1
            else:
                table[b, j] = -1
                lacking += 1
        for p in range(c, c + n):
            block = table[b, p // bs] if p // bs < width else -1
            pos.append(p)
            rows.append(b)
            slots.append(int(block) * bs + p % bs if block >= 0 else -1)
        offsets.append(offsets[-1] + n)
    more = max(N - len(pos), 0)
    return (table, offsets, (pos + [0] * more)[:N], (slots + [-1] * more)[:N],
            (rows + [-1] * more)[:N], [taken, lacking])


def check(jet, cached, added, bs, table, free, nxt, N):
    dev = lambda a, t: torch.tensor(np.asarray(a), dtype=t).cuda()
    t = dev(table, torch.int32)
    out = jet.kv_slot_map(dev(cached, torch.int32), dev(added, torch.int32), bs, t,
                          dev(free, torch.int32), dev([nxt], torch.int64), N)
    torch.cuda.synchronize()
    want = plain(np.asarray(cached), np.asarray(added), bs, np.asarray(table), list(free), nxt, N)
    assert np.array_equal(t.cpu().numpy(), want[0])
    for name, got, ref in zip(("offsets", "positions", "slots", "rows", "counts"), out, want[1:]):
        assert got.tolist() == list(ref), name
    return out


def state(rng, B, most_cached, most_added, bs, spare=5):
    cached = rng.integers(0, most_cached + 1, B)
    added = rng.integers(0, most_added + 1, B)
    old, new = -(-cached // bs), -(-(cached + added) // bs)
    width = int(-(-(most_cached + most_added) // bs)) or 1
    ids = rng.permutation(int(new.sum()) + spare).astype(np.int32)
    table, at = np.full((B, width), -1, np.int32), 0
    for b in range(B):
        table[b, :old[b]] = ids[at:at + old[b]]
        at += old[b]
    return cached, added, table, ids[at:]


@pytest.mark.parametrize("B,most_cached,most_added,bs", [
    (1, 0, 1, 16), (1, 100, 1, 16), (3, 40, 9, 4), (256, 300, 1, 16), (48, 500, 200, 64), (513, 40, 3, 8),
    (1030, 20, 2, 1), (7, 1000, 700, 24), (2, 5, 3000, 7), (2457, 6, 2, 4), (5000, 10, 1, 3), (8192, 3, 1, 2)])
@pytest.mark.parametrize("extra", [0, 37])
def test_against_the_loop(jet, B, most_cached, most_added, bs, extra):
    rng = np.random.default_rng(B + bs)
    cached, added, table, free = state(rng, B, most_cached, most_added, bs)
    check(jet, cached, added, bs, table, free, 0, int(added.sum()) + extra)


def test_free_list_position_and_shortage(jet):
    rng = np.random.default_rng(3)
    cached, added, table, free = state(rng, 20, 50, 60, 8)
    check(jet, cached, added, 8, table, np.concatenate([[7, 7, 7], free]), 3, 1500)
    for n in (0, 1, len(free) // 2):
        out = check(jet, cached, added, 8, table, free[:n], 0, 1500)
        assert int(out[4][1]) > 0
    check(jet, cached, added, 8, table, free, len(free) + 9, 1500)      # past the list's end: none left
    check(jet, cached, added, 8, table, free, -4, 1500)


def test_narrow_table_small_capacity_and_bad_lengths(jet):
    rng = np.random.default_rng(4)
    cached, added, table, free = state(rng, 9, 30, 90, 8)
    check(jet, cached, added, 8, np.ascontiguousarray(table[:, :5]), free, 0, 700)   # tokens past the width
    total = int(added.sum())
    check(jet, cached, added, 8, table, free, 0, total // 3)             # outputs cut, the table complete
    check(jet, cached, added, 8, table, free, 0, 0)
    cached[2], added[5] = -7, -3                                         # counted as none
    table[2] = -1
    check(jet, cached, added, 8, table, np.arange(100, 600), 0, 700)
    table[4, 0] = -1                                                     # a hole behind cached tokens
    check(jet, cached, added, 8, table, np.arange(100, 600), 0, 700)


def test_no_request(jet):
    e = np.zeros((0,), np.int32)
    check(jet, e, e, 16, np.zeros((0, 4), np.int32), [1, 2, 3], 1, 5)


def test_steps_of_a_decoding_loop(jet):
    """Three steps, each call's counts the next one's free_next; the slots of
    all steps are distinct and the cache write takes them."""
    B, bs, S = 17, 4, 64
    rng = np.random.default_rng(8)
    cached = torch.tensor(rng.integers(0, 6, B), dtype=torch.int32).cuda()
    table = torch.full((B, 4), -1, dtype=torch.int32, device="cuda")
    free = torch.tensor(rng.permutation(S), dtype=torch.int32).cuda()
    nxt = torch.zeros((1,), dtype=torch.int64, device="cuda")
    _, _, _, _, counts = jet.kv_slot_map(torch.zeros_like(cached), cached, bs, table, free, nxt, 128)
    seen = []
    ones = torch.ones_like(cached)
    cache = torch.zeros((S * bs, 2, 16), dtype=torch.uint8, device="cuda")
    scale = torch.ones((2,), device="cuda")
    for step in range(3):
        _, pos, slots, rows, counts = jet.kv_slot_map(cached, ones, bs, table, free, counts[:1], B)
        x = torch.full((B, 2, 16), float(step + 1), device="cuda").to(torch.bfloat16)
        jet.jet_kv_cache_write(x, scale, slots, cache)
        assert pos.tolist() == cached.tolist() and rows.tolist() == list(range(B))
        seen += slots.tolist()
        cached += 1
    assert min(seen) >= 0 and len(set(seen)) == 3 * B
    assert int((cache != 0).any(2).any(1).sum()) == 3 * B
