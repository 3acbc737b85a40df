"""spec_tree_rows and spec_kv_append against their definitions in 64 bits (needs an MI355X)."""
import math

import numpy as np
import pytest
import torch

from lossless_speculative_sampling_amd import capi

pytestmark = pytest.mark.gpu
DT = {"bf16": torch.bfloat16, "fp16": torch.float16}


def tree_oracle(tokens, parents, slots, ctx, depth):
    B, N = tokens.shape
    pos, app, ln = np.full((B, N), -1), np.full((B, N), -1), np.zeros((B, N), int)
    lists = np.full((B, N, depth), -1)
    for b in range(B):
        paths = {}
        for n in range(N):
            p = parents[b, n]
            if tokens[b, n] < 0 or p < -1 or p >= n or (p >= 0 and p not in paths):
                continue
            path = (paths[p] if p >= 0 else []) + [slots[b, n]]
            if len(path) > depth:
                continue
            paths[n] = path
            pos[b, n], app[b, n], ln[b, n] = ctx[b] + len(path) - 1, slots[b, n], len(path)
            lists[b, n, :len(path)] = path
    return pos, app, lists, ln


@pytest.mark.parametrize("B,N,depth", [(1, 1, 1), (3, 2, 1), (2, 37, 6), (5, 100, 16), (2, 300, 300), (1, 4096, 9), (2, 4097, 12),
                                       (300, 64, 8)])
def test_tree_rows(B, N, depth):
    rng = np.random.default_rng(B + N)
    tokens = rng.integers(0, 1000, (B, N))
    parents = np.where(rng.random((B, N)) < 0.4, np.arange(N) - 1, [[int(rng.integers(-1, max(n, 1))) for n in range(N)] for _ in range(B)])
    tokens[rng.random((B, N)) < 0.03] = -1
    odd = rng.random((B, N)) < 0.02
    parents[odd] = rng.choice([-2, N, N + 5, -(1 << 31), (1 << 31) - 1], int(odd.sum()))
    if N > 3:
        parents[0, 3] = 3  # its own parent
    slots, ctx = rng.integers(0, 1 << 30, (B, N)), rng.integers(0, 1 << 20, B)
    want = tree_oracle(tokens, parents, slots, ctx, depth)
    dev = [torch.as_tensor(x.astype(np.int32)).cuda() for x in (tokens, parents, slots, ctx)]
    print(f"[rows] B={B} N={N} depth={depth}", flush=True)
    r = capi.spec_tree_rows(*dev, depth)
    for got, ref in zip((r.positions, r.append_slots, r.suffix_slots, r.suffix_len), want):
        np.testing.assert_array_equal(got.cpu().numpy(), ref)


def rotated(x, positions, freqs, scale, interleaved):
    """float64 rotation of x [T][h][D]."""
    rot = 2 * len(freqs)
    y = x.double().clone()
    ang = positions.double()[:, None, None] * torch.as_tensor(freqs, dtype=torch.float64)
    c, s = torch.cos(ang) * scale, torch.sin(ang) * scale
    a, b = (slice(0, rot, 2), slice(1, rot, 2)) if interleaved else (slice(0, rot // 2), slice(rot // 2, rot))
    y[..., a], y[..., b] = x.double()[..., a] * c - x.double()[..., b] * s, x.double()[..., b] * c + x.double()[..., a] * s
    return y


def near(got, want, size, dtype):
    """One rounding to dtype (half a step of the value, at the subnormals half of the smallest), after fp32 sums
    whose angle is off by up to 2^-22 of the pair's length."""
    info = torch.finfo(dtype)
    off = (got.double() - want).abs()
    bound = info.eps / 2 * want.abs() + info.smallest_normal * info.eps / 2 + size * 2.0 ** -21
    assert (off <= bound).all(), (off - bound).max()


def make(T, Hq, Hkv, D, dtype, cache, page, seed, pages=None):
    g = torch.Generator().manual_seed(seed)
    pages = pages or (2 * T // page + 2)
    x = [torch.randn((T, h, D), generator=g).to(dtype).cuda() for h in (Hq, Hkv, Hkv)]
    kc, vc = (torch.randn((pages, page, Hkv, D), generator=g).to(cache).cuda() for _ in range(2))
    return (*x, kc, vc)


CASES = [  # T, Hq, Hkv, D, rot, interleaved, dtype, e4m3, page, far
    (1, 1, 1, 8, 8, True, "bf16", False, 1, 10), (3, 4, 2, 64, 64, False, "bf16", False, 16, 1000),
    (5, 6, 2, 64, 64, True, "fp16", False, 16, 100000), (7, 8, 1, 128, 64, False, "bf16", True, 32, 1 << 20),
    (9, 3, 3, 80, 40, False, "fp16", False, 7, 5000), (4, 2, 2, 80, 40, True, "bf16", True, 7, 5000),
    (2, 5, 1, 33, 10, False, "bf16", False, 3, 77), (3, 2, 2, 15, 14, True, "fp16", True, 4, 77),
    (6, 4, 4, 96, 0, False, "bf16", False, 16, 3), (300, 8, 2, 256, 256, False, "bf16", False, 64, 1 << 24),
    (257, 4, 1, 128, 128, True, "fp16", True, 128, (1 << 31) - 1)]


@pytest.mark.parametrize("T,Hq,Hkv,D,rot,inter,dt,eight,page,far", CASES)
def test_append(T, Hq, Hkv, D, rot, inter, dt, eight, page, far):
    dtype = DT[dt]
    rng = np.random.default_rng(T * D + rot)
    q, k, v, kc, vc = make(T, Hq, Hkv, D, dtype, torch.float8_e4m3fn if eight else dtype, page, T + D)
    before = [kc.clone(), vc.clone()]
    total = kc.shape[0] * page
    slots = rng.permutation(total)[:T]
    if T > 2:
        slots[T // 2] = -1
    bad = T > 4
    if bad:
        slots[1], slots[3] = total, -2
    positions = rng.integers(-5 if far < 100 else 0, far, T)
    positions[-1] = far - 1
    scales = [0.25 + torch.rand(Hkv, device="cuda") for _ in range(2)] if eight else [None, None]
    freqs = capi.spec_rope_frequencies(rot, base=500000.0, factor=8.0) if rot else []
    rotary = capi.Rotary(torch.tensor(freqs, dtype=torch.float64, device="cuda"), interleaved=inter, scale=1.25) if rot else None
    dev = [torch.as_tensor(x.astype(np.int32)).cuda() for x in (positions, slots)]
    status = torch.full((T,), 7, dtype=torch.int32, device="cuda")
    print(f"[append] T={T} D={D} rot={rot} {dt} e4m3={eight}", flush=True)
    got = capi.spec_kv_append(k, v, dev[0], dev[1], capi.KVCache(kc, vc, *scales), rotary, q=q, status=status)
    pos = torch.as_tensor(positions)
    length = lambda x: x.double().abs().amax(-1, keepdim=True) * 1.25 * math.sqrt(2) * (rot > 0)  # noqa: E731
    near(got.cpu(), rotated(q.cpu(), pos, freqs, 1.25, inter), length(q.cpu()), dtype)
    ok = (slots >= 0) & (slots < total)
    want = (slots >= total) | (slots < -1)
    np.testing.assert_array_equal(status.cpu().numpy(), want * capi.ST_BAD_SLOT)
    for x, cache, old, scale, turns in ((k, kc, before[0], scales[0], True), (v, vc, before[1], scales[1], False)):
        now, was = cache.cpu().view(-1, Hkv, D), old.cpu().view(-1, Hkv, D)
        idle = np.setdiff1d(np.arange(total), slots[ok])
        raw = torch.uint8 if eight else torch.int16
        assert torch.equal(now.view(raw)[idle], was.view(raw)[idle]), "a slot that was not named changed"
        ref = rotated(x.cpu(), pos, freqs, 1.25, inter) if turns else x.cpu().double()
        size = length(x.cpu()) if turns else torch.zeros(T, 1, 1, dtype=torch.float64)
        if eight:
            by = scale.cpu().double()[:, None]
            ref, size = (ref / by).clamp(-448, 448), size / by
            near(now[slots[ok]].float(), ref[ok], size[ok] + ref[ok].abs() * 2.0 ** -3, torch.float8_e4m3fn)
        elif turns and rot:
            near(now[slots[ok]], ref[ok], size[ok], dtype)
        else:
            assert torch.equal(now[slots[ok]], x.cpu()[ok])


def test_e4m3_rounding_and_range():
    """Every e4m3 value, the middles between neighbours (ties to even), both ends, NaN and zeros."""
    every = torch.arange(256, dtype=torch.int32).to(torch.uint8).view(torch.float8_e4m3fn).float()
    fin = every[torch.isfinite(every)].unique()
    mid = (fin[1:] + fin[:-1]) / 2
    x = torch.cat([fin, mid, torch.tensor([1e4, -1e4, 448.0, 460.0, 464.0, -500.0, float("inf"), float("-inf"), float("nan"), -0.0, 2 ** -10, -2 ** -10])])
    x = torch.cat([x, torch.zeros(-len(x) % 16)]).to(torch.float16)
    T = len(x) // 16
    v = x.view(T, 2, 8).cuda()
    kc = torch.zeros((T, 1, 2, 8), device="cuda").to(torch.float8_e4m3fn)
    vc = torch.zeros_like(kc)
    capi.spec_kv_append(v, v, None, torch.arange(T, dtype=torch.int32, device="cuda"), capi.KVCache(kc, vc))
    want = v.cpu().float()
    want = torch.where(want.isnan(), want, want.clamp(-448, 448)).to(torch.float8_e4m3fn)
    for c in (kc, vc):
        a, b = c.cpu().view(T, 2, 8).float(), want.float()
        assert torch.equal(a.isnan(), b.isnan()) and torch.equal(a.nan_to_num(7), b.nan_to_num(7))


def test_strided_views_in_place_and_queries_alone():
    T, Hq, Hkv, D, page = 9, 4, 2, 64, 8
    g = torch.Generator().manual_seed(0)
    qkv = torch.randn((T, Hq + 2 * Hkv, D), generator=g).to(torch.bfloat16).cuda()  # one projection's output
    q, k, v = qkv[:, :Hq], qkv[:, Hq:Hq + Hkv], qkv[:, Hq + Hkv:]
    both = torch.zeros((4, 2, Hkv, page, D), dtype=torch.bfloat16, device="cuda")  # keys and values side by side, heads outside
    cache = capi.KVCache(both[:, 0].transpose(1, 2), both[:, 1].transpose(1, 2))
    freqs = capi.spec_rope_frequencies(D)
    rotary = capi.Rotary(torch.tensor(freqs, dtype=torch.float64, device="cuda"))
    pos, slots = torch.arange(100, 100 + T, dtype=torch.int32, device="cuda"), torch.randperm(4 * page, generator=g)[:T].to(torch.int32).cuda()
    plain = capi.KVCache(torch.zeros((4, page, Hkv, D), dtype=torch.bfloat16, device="cuda"), torch.zeros((4, page, Hkv, D), dtype=torch.bfloat16, device="cuda"))
    ref = capi.spec_kv_append(k.contiguous(), v.contiguous(), pos, slots, plain, rotary, q=q.contiguous())
    alone = capi.spec_kv_append(None, None, pos, None, None, rotary, q=q)
    assert torch.equal(alone, ref)
    got = capi.spec_kv_append(k, v, pos, slots, cache, rotary, q=q, q_out=q)  # in place
    assert got.data_ptr() == q.data_ptr() and torch.equal(q, ref)
    assert torch.equal(cache.k, plain.k) and torch.equal(cache.v, plain.v)
    near(ref.cpu(), rotated(torch.randn((T, Hq + 2 * Hkv, D), generator=torch.Generator().manual_seed(0)).to(torch.bfloat16)[:, :Hq], pos.cpu(), freqs, 1.0, False), 8.0, torch.bfloat16)
    # one element off the vectors' alignment: the same values
    odd = torch.zeros(T * (Hq + 2 * Hkv) * D + 1, dtype=torch.bfloat16, device="cuda")[1:].view(T, Hq + 2 * Hkv, D)
    odd.copy_(torch.randn((T, Hq + 2 * Hkv, D), generator=torch.Generator().manual_seed(0)).to(torch.bfloat16))
    other = capi.KVCache(torch.zeros_like(plain.k), torch.zeros_like(plain.v))
    assert torch.equal(capi.spec_kv_append(odd[:, Hq:Hq + Hkv], odd[:, Hq + Hkv:], pos, slots, other, rotary, q=odd[:, :Hq]), ref)
    assert torch.equal(other.k, plain.k) and torch.equal(other.v, plain.v)
    # no tokens at all
    assert capi.spec_kv_append(k[:0], v[:0], pos[:0], slots[:0], cache, rotary, q=q[:0]).shape == (0, Hq, D)


def test_named_streams_graphs_and_outputs_given():
    T, Hq, Hkv, D, page = 40, 4, 2, 64, 16
    q, k, v, kc, vc = make(T, Hq, Hkv, D, torch.bfloat16, torch.bfloat16, page, 3)
    rotary = capi.Rotary(torch.tensor(capi.spec_rope_frequencies(D), dtype=torch.float64, device="cuda"), interleaved=True)
    g = torch.Generator().manual_seed(5)
    pos = torch.randint(0, 9999, (T,), generator=g, dtype=torch.int32).cuda()
    slots = torch.randperm(kc.shape[0] * page, generator=g)[:T].to(torch.int32).cuda()
    tok, par = torch.randint(0, 9, (3, 50), generator=g, dtype=torch.int32).cuda(), (torch.arange(50, dtype=torch.int32) - 1).expand(3, 50).contiguous().cuda()
    node, ctx = torch.randint(0, 999, (3, 50), generator=g, dtype=torch.int32).cuda(), torch.tensor([0, 7, 500], dtype=torch.int32, device="cuda")
    ref = capi.spec_kv_append(k, v, pos, slots, capi.KVCache(kc, vc), rotary, q=q)
    rows = capi.spec_tree_rows(tok, par, node, ctx, 50)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    for stream in (s, s.cuda_stream):
        c2 = capi.KVCache(kc.clone(), vc.clone())
        torch.cuda.synchronize()
        got = capi.spec_kv_append(k, v, pos, slots, c2, rotary, q=q, stream=stream)
        r2 = capi.spec_tree_rows(tok, par, node, ctx, 50, stream=stream)
        s.synchronize()
        assert torch.equal(got, ref) and torch.equal(c2.k, kc) and torch.equal(c2.v, vc)
        assert torch.equal(r2.suffix_slots, rows.suffix_slots) and torch.equal(r2.positions, rows.positions)
    held = capi.KVCache(torch.zeros_like(kc), torch.zeros_like(vc))
    out = torch.empty_like(q)
    trees = capi.TreeRows(*[torch.empty_like(x) for x in (rows.positions, rows.append_slots, rows.suffix_slots, rows.suffix_len)])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        capi.spec_kv_append(k, v, pos, slots, held, rotary, q=q, q_out=out)
        capi.spec_tree_rows(tok, par, node, ctx, 50, out=trees)
    for i in range(4):
        k.normal_()
        pos.add_(13)
        ctx.add_(1)
        graph.replay()
        torch.cuda.synchronize()
        now = capi.KVCache(torch.zeros_like(kc), torch.zeros_like(vc))
        want = capi.spec_kv_append(k, v, pos, slots, now, rotary, q=q)
        assert torch.equal(out, want) and torch.equal(held.k, now.k) and torch.equal(held.v, now.v)
        r2 = capi.spec_tree_rows(tok, par, node, ctx, 50)
        assert torch.equal(trees.positions, r2.positions) and torch.equal(trees.suffix_slots, r2.suffix_slots)


def test_offsets_past_32_bits():
    """A cache of more than 2^32 elements: the last slots are written where they belong."""
    Hkv, D, page = 8, 128, 64
    pages = (1 << 32) // (page * Hkv * D) + 3
    kc = torch.zeros((pages, page, Hkv, D), dtype=torch.bfloat16, device="cuda")
    vc = torch.zeros_like(kc)
    k, v = (torch.randn((3, Hkv, D), device="cuda").to(torch.bfloat16) for _ in range(2))
    slots = torch.tensor([pages * page - 1, 0, (pages - 2) * page + 5], dtype=torch.int32, device="cuda")
    capi.spec_kv_append(k, v, None, slots, capi.KVCache(kc, vc))
    s = slots.long()
    assert torch.equal(kc.view(-1, Hkv, D)[s], k) and torch.equal(vc.view(-1, Hkv, D)[s], v)
    assert int((kc.view(-1, Hkv * D)[:, 0] != 0).sum()) <= 3
