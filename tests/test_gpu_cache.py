"""Paged cache on the GPU: the store of new tokens, and the attention of one
new token of each sequence, against 64 bits."""
import pytest
import torch

import block_ref as ref

pytestmark = pytest.mark.gpu
KINDS = ref.KINDS


# ---------------------------------------------------------------------------
# store
# ---------------------------------------------------------------------------
@pytest.mark.parametrize("kind", ["f16", "bf16"])
@pytest.mark.parametrize("d", [8, 40, 64, 128])
@pytest.mark.parametrize("kv,page,n", [(1, 1, 1), (2, 16, 37), (8, 16, 200), (3, 24, 50), (1, 64, 300)])
def test_store(lib, kv, page, n, d, kind):
    from post_weight_quantization_04_amd import layer
    kind = KINDS[kind]
    gen = torch.Generator().manual_seed(n + d)
    pages = -(-n // page) + 5
    cache = layer.kv_cache(pages, kv, page, d, kind)
    before = [torch.randn(pages, kv, page, d, generator=gen).to(kind) for _ in range(2)]
    cache.keys.copy_(before[0])
    cache.values.copy_(before[1])
    k, v = (torch.randn(n, kv, d, generator=gen).to(kind) for _ in range(2))
    slots = torch.randperm(pages * page, generator=gen)[:n].to(torch.int32)
    slots[::7] = -1                       # padding
    slots[3::11] = pages * page + 4       # outside
    layer.cache_store(cache, k.cuda(), v.cuda(), slots.cuda())
    for new, old, got in ((k, before[0], cache.keys), (v, before[1], cache.values)):
        want = old.clone()
        for t, s in enumerate(slots.tolist()):
            if 0 <= s < pages * page:
                want[s // page, :, s % page] = new[t]
        assert torch.equal(got.cpu(), want)


def test_store_strides(lib):
    """Rows first in the cache, views of a fused projection, keys and values in one tensor."""
    from post_weight_quantization_04_amd import layer
    pages, kv, page, d, n = 9, 3, 16, 64, 70
    both = torch.zeros(2, pages, page, kv, d, dtype=torch.float16, device="cuda")
    cache = layer.KVCache(both[0].transpose(1, 2), both[1].transpose(1, 2))
    fused = torch.randn(n, 2 * kv * d).half().cuda()
    k, v = (t.view(n, kv, d) for t in fused.split(kv * d, dim=1))
    slots = torch.randperm(pages * page)[:n].to(torch.int32).cuda()
    layer.cache_store(cache, k, v, slots)
    want = torch.zeros_like(both)
    want[0].view(-1, kv, d)[slots.long()] = k
    want[1].view(-1, kv, d)[slots.long()] = v
    assert torch.equal(both, want)


def test_store_nothing(lib):
    from post_weight_quantization_04_amd import layer
    cache = layer.kv_cache(4, 2, 16, 64)
    cache.keys.zero_(), cache.values.zero_()
    k = torch.ones(3, 2, 64, dtype=torch.float16, device="cuda")
    slots = torch.full((3,), -1, dtype=torch.int32, device="cuda")
    layer.cache_store(cache, k, k, slots)
    layer.cache_store(cache, k[:0], k[:0], slots[:0])
    assert not bool(cache.keys.any()) and not bool(cache.values.any())


# ---------------------------------------------------------------------------
# attention
# ---------------------------------------------------------------------------
def make(lengths, heads, kv, d, page, kind, seed=0, spare=3, sharp=1.0):
    """q, keys, values, table, lengths: pages in no order, NaN in everything that no sequence holds."""
    gen = torch.Generator().manual_seed(seed)
    used = [-(-v // page) for v in lengths]
    pages, most = sum(used) + spare, max(used + [0])
    order = torch.randperm(pages, generator=gen)
    table = torch.full((len(lengths), most), -1, dtype=torch.int32)
    keys = torch.full((pages, kv, page, d), float("nan"), dtype=kind)
    values = torch.full((pages, kv, page, d), float("nan"), dtype=kind)
    at = 0
    for b, length in enumerate(lengths):
        table[b, :used[b]] = order[at:at + used[b]].to(torch.int32)
        at += used[b]
        for i in range(used[b]):
            rows = min(page, length - i * page)
            keys[table[b, i], :, :rows] = torch.randn(kv, rows, d, generator=gen).to(kind)
            values[table[b, i], :, :rows] = torch.randn(kv, rows, d, generator=gen).to(kind)
    q = (torch.randn(len(lengths), heads, d, generator=gen) * sharp).to(kind)
    return q, keys, values, table, torch.tensor(lengths, dtype=torch.int32)


def call(q, keys, values, table, lengths, **more):
    from post_weight_quantization_04_amd import layer
    return layer.cached_attention(q.cuda(), layer.KVCache(keys.cuda(), values.cuda()), table.cuda(), lengths.cuda(), **more)


def check(lengths, heads, kv, d, page, kind, scale=None, seed=0, sharp=1.0):
    kind = KINDS[kind]
    case = make(lengths, heads, kv, d, page, kind, seed, sharp=sharp)
    got = call(*case, scale=scale)
    want, off = ref.cached(*case, d ** -0.5 if scale is None else scale, kind)
    ref.near(got, want, off, f"{lengths} {heads}/{kv} x {d}, pages of {page}")


@pytest.mark.parametrize("kind", ["f16", "bf16"])
@pytest.mark.parametrize("page", [1, 3, 16, 24, 64, 100])
@pytest.mark.parametrize("n", [0, 1, 2, 15, 16, 17, 31, 32, 33, 63, 64, 65, 127, 128, 129, 300])
def test_lengths(lib, n, page, kind):
    check([n], 4, 2, 64, page, kind, seed=n)


@pytest.mark.parametrize("d", [8, 16, 24, 40, 56, 64, 72, 80, 96, 120, 128])
def test_head_sizes(lib, d):
    check([70, 0, 3, 129], 4, 2, d, 16, "f16", seed=d)
    check([33, 140], 3, 3, d, 24, "bf16", seed=d)


@pytest.mark.parametrize("heads,kv", [(1, 1), (2, 1), (3, 1), (4, 4), (5, 1), (6, 2), (7, 1), (8, 1), (12, 4), (16, 1),
                                      (16, 2), (24, 2), (17, 1), (33, 1), (40, 2)])
@pytest.mark.parametrize("d", [64, 128])
def test_heads_that_share_keys(lib, heads, kv, d):
    check([45, 300, 1], heads, kv, d, 16, "f16", seed=heads)


@pytest.mark.parametrize("lengths", [[0, 0, 0], [0, 5, 0, 700, 0], [1] * 70, [1, 2000, 1, 3], list(range(40)),
                                     [511, 512, 513], [1024, 64, 4096]])
def test_ragged(lib, lengths):
    check(lengths, 4, 2, 64, 16, "f16")
    check(lengths, 8, 1, 128, 32, "bf16")


@pytest.mark.parametrize("kind", ["f16", "bf16"])
@pytest.mark.parametrize("sharp,scale", [(8.0, None), (1.0, 0.01), (1.0, 3.0), (30.0, 1.0)])
def test_scales(lib, kind, sharp, scale):
    check([150, 1700], 2, 1, 64, 16, kind, scale, sharp=sharp)


def test_long(lib):
    check([20000], 4, 1, 128, 64, "bf16")
    check([9000, 3, 15000], 2, 2, 64, 16, "f16")


def test_pages_that_are_gone(lib):
    """Page numbers outside the cache: their tokens are masked; a sequence of none but those gives zeros."""
    for seed in range(3):
        q, keys, values, table, lengths = make([200, 90, 40, 700], 4, 2, 64, 16, torch.float16, seed)
        table[0, 2], table[0, 12], table[1, 0], table[1, 5] = -1, 1 << 30, -7, keys.shape[0]
        table[2, :] = -1
        table[3, 3:30] = -1
        got = call(q, keys, values, table, lengths)
        want, off = ref.cached(q, keys, values, table, lengths, 64 ** -0.5, torch.float16)
        assert not bool(got[2].any())
        ref.near(got, want, off)


def test_lengths_that_leave_the_table(lib):
    q, keys, values, table, _ = make([48, 48], 4, 2, 64, 16, torch.float16)
    got = call(q, keys, values, table, torch.tensor([1 << 30, -3], dtype=torch.int32))
    want = call(q, keys, values, table, torch.tensor([48, 0], dtype=torch.int32))
    assert torch.equal(got, want) and not bool(got[1].any())


def test_a_shared_page(lib):
    """Two sequences that begin alike share pages; one of them twice in its own table."""
    q, keys, values, table, lengths = make([100, 64], 4, 2, 64, 16, torch.float16)
    table[1, :2] = table[0, :2]
    table[1, 3] = table[1, 2]
    got = call(q, keys, values, table, lengths)
    want, off = ref.cached(q, keys, values, table, lengths, 64 ** -0.5, torch.float16)
    ref.near(got, want, off)


def test_seen_infinities(lib):
    """An infinite value that is seen reaches its own column; a NaN key its whole row; neither another sequence."""
    case = make([70, 50, 600], 4, 2, 64, 16, torch.bfloat16)
    clean = call(*case).cpu()
    q, keys, values, table, lengths = case
    values[table[2, 20], 1, 3, 9] = float("inf")
    keys[table[1, 1], 0, 2, 5] = float("nan")
    got = call(q, keys, values, table, lengths).cpu()
    assert torch.equal(got[0], clean[0]) and torch.equal(got[2, :2], clean[2, :2]) and torch.equal(got[1, 2:], clean[1, 2:])
    assert torch.isnan(got[1, :2]).all()
    assert bool((got[2, 2:, 9] == float("inf")).all())
    other = [c for c in range(64) if c != 9]
    assert torch.equal(got[2, 2:][:, other], clean[2, 2:][:, other])


def test_strides(lib):
    """Rows before heads in the cache, a wider table, q inside a fused projection."""
    from post_weight_quantization_04_amd import layer
    q, keys, values, table, lengths = make([77, 300], 6, 2, 64, 16, torch.float16)
    want = call(q, keys, values, table, lengths)
    turned = [t.transpose(1, 2).contiguous().cuda().transpose(1, 2) for t in (keys, values)]
    wide = torch.full((2, table.shape[1] + 5), 1 << 29, dtype=torch.int32)
    wide[:, :table.shape[1]] = table
    fused = torch.zeros(2, 10 * 64, dtype=torch.float16)
    fused[:, :6 * 64] = q.view(2, -1)
    out = torch.full((2, 8, 64), 7.0, dtype=torch.float16, device="cuda")
    layer.cached_attention(fused.cuda()[:, :6 * 64].view(2, 6, 64), layer.KVCache(*turned),
                           wide.cuda()[:, :table.shape[1]], lengths.cuda(), out=out[:, :6])
    assert torch.equal(out[:, :6], want) and bool((out[:, 6:] == 7.0).all())


def test_workspace(lib):
    """One workspace for calls of many sizes, whatever it held before."""
    from post_weight_quantization_04_amd import layer
    ws = layer.Workspace()
    for lengths in ([3000], [5, 900], [70] * 30, [1]):
        case = make(lengths, 8, 2, 64, 16, torch.float16)
        want = call(*case)
        if ws.buf is not None:
            ws.buf.fill_(255)
        assert torch.equal(call(*case, ws=ws), want)


def test_a_captured_call_follows_its_lengths(lib):
    from post_weight_quantization_04_amd import layer
    q, keys, values, table, lengths = (t.cuda() for t in make([500, 900, 64], 4, 2, 64, 16, torch.float16))
    cache, ws, out = layer.KVCache(keys, values), layer.Workspace(), torch.empty_like(q)
    layer.cached_attention(q, cache, table, lengths, ws=ws, out=out)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        layer.cached_attention(q, cache, table, lengths, ws=ws, out=out)
    for now in ([500, 900, 64], [1, 0, 64], [499, 17, 3], [0, 0, 0], [300, 899, 63]):
        lengths.copy_(torch.tensor(now, dtype=torch.int32))
        out.fill_(9.0)
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, layer.cached_attention(q, cache, table, lengths))


def test_two_streams_at_once(lib):
    """Calls at the same time, each with scratch memory of its own."""
    from post_weight_quantization_04_amd import layer
    a = [t.cuda() for t in make([4000, 70], 8, 2, 128, 16, torch.float16, 1)]
    b = [t.cuda() for t in make([300, 5000], 8, 2, 128, 16, torch.float16, 2)]
    run = lambda c, **m: layer.cached_attention(c[0], layer.KVCache(c[1], c[2]), c[3], c[4], **m)  # noqa: E731
    want = run(a), run(b)
    sides = [torch.cuda.Stream() for _ in range(2)]
    for s in sides:
        s.wait_stream(torch.cuda.current_stream())
    got = [[run(c, stream=s) for c, s in zip((a, b), sides)] for _ in range(4)]
    torch.cuda.synchronize()
    assert all(torch.equal(g[0], want[0]) and torch.equal(g[1], want[1]) for g in got)


def test_deterministic(lib):
    case = make([3000, 20, 700], 8, 2, 128, 16, torch.float16)
    first = call(*case)
    assert all(torch.equal(call(*case), first) for _ in range(3))


def test_empty(lib):
    q, keys, values, table, lengths = make([40, 3], 4, 2, 64, 16, torch.float16)
    assert call(q[:0], keys, values, table[:0], lengths[:0]).shape == (0, 4, 64)
    assert not bool(call(q, keys, values, table[:, :0], lengths).any())
    assert not bool(call(q, keys[:0], values[:0], table, lengths).any())


@pytest.mark.parametrize("d", [64, 128])
def test_more_units_than_compute_units(lib, d):
    """Many sequences, in tables of up to 1024 tokens and in longer ones (divided and joined)."""
    short = [(37 * i) % 190 for i in range(150)]
    check(short, 4, 2, d, 16, "f16")
    check(short + [2100, 0, 1], 4, 2, d, 16, "bf16")


def test_a_cache_past_32_bits(lib):
    """Pages whose offsets do not fit 32 bits, in elements and in bytes."""
    from post_weight_quantization_04_amd import layer
    kv, page, d, pages = 8, 64, 128, 33000
    assert pages * kv * page * d > 1 << 31
    cache = layer.kv_cache(pages, kv, page, d)
    gen = torch.Generator().manual_seed(5)
    lengths = [130, 1500, 64]
    n = sum(lengths)
    k, v = (torch.randn(n, kv, d, generator=gen).half() for _ in range(2))
    used = [-(-x // page) for x in lengths]
    table = torch.zeros(3, max(used), dtype=torch.int32)
    far = pages - 1
    for b in range(3):
        for i in range(used[b]):
            table[b, i] = far if i % 2 else 3 + far % 1000
            far -= 1
    slots = torch.cat([table[b, torch.arange(x) // page] * page + torch.arange(x) % page for b, x in enumerate(lengths)])
    layer.cache_store(cache, k.cuda(), v.cuda(), slots.to(torch.int32).cuda())
    q = torch.randn(3, 32, d, generator=gen).half()
    got = layer.cached_attention(q.cuda(), cache, table.cuda(), torch.tensor(lengths, dtype=torch.int32).cuda())
    # the same tokens in a small cache
    small = torch.arange(sum(used), dtype=torch.int32)
    rows, at, t = torch.zeros_like(table), 0, 0
    keys, values = (torch.zeros(sum(used), kv, page, d, dtype=torch.float16) for _ in range(2))
    for b, x in enumerate(lengths):
        rows[b, :used[b]] = small[at:at + used[b]]
        for j in range(x):
            keys[at + j // page, :, j % page], values[at + j // page, :, j % page] = k[t + j], v[t + j]
        at, t = at + used[b], t + x
    assert torch.equal(got, call(q, keys, values, rows, torch.tensor(lengths, dtype=torch.int32)))
