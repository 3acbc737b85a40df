"""spec_prefix_attention against its definition in 64 bits (needs an MI355X)."""
import math

import numpy as np
import pytest
import torch

from lossless_speculative_sampling_amd import capi

pytestmark = pytest.mark.gpu
DT = {"bf16": torch.bfloat16, "fp16": torch.float16, "e4m3": torch.float8_e4m3fn}


class Case:
    """One batch: groups of rows, paged prefixes, suffix lists."""

    def __init__(self, rows, prefix, suffix, Hq, Hkv, D, dtype="bf16", cache=None, page=16, seed=0, pad=0, size=1.0, spare=2):
        g = torch.Generator().manual_seed(seed)
        rng = np.random.default_rng(seed)
        self.G, self.R = len(rows), int(sum(rows)) + pad
        self.Hq, self.Hkv, self.D, self.page, self.pad = Hq, Hkv, D, page, pad
        self.dtype, cdt = DT[dtype], DT[cache or dtype]
        self.prefix, self.start = np.array(prefix), np.concatenate([[0], np.cumsum(rows)])
        wide = max(1, -(-max(prefix) // page)) + 1  # one column more than needed
        S = max(1, int(max(suffix)))
        self.lens = np.resize(np.array(suffix), self.R)
        spots = self.R * S + 3
        extra = -(-spots // page)
        pages = self.G * wide + extra + spare
        order = rng.permutation(pages)
        self.table = order[:self.G * wide].reshape(self.G, wide)
        slots = (order[self.G * wide:self.G * wide + extra, None] * page + np.arange(page)).reshape(-1)
        self.lists = rng.permutation(slots)[:self.R * S].reshape(self.R, S)
        self.q = (torch.randn((self.R, Hq, D), generator=g) * size).to(self.dtype)
        self.k, self.v = (torch.randn((pages, page, Hkv, D), generator=g).to(cdt) for _ in range(2))
        self.scales = [0.5 + torch.rand(Hkv, generator=g) for _ in range(2)] if cdt == DT["e4m3"] else [None, None]
        self.scale = D ** -0.5
        self.name = f"rows={list(rows)} prefix={list(prefix)} suffix={list(suffix)} H={Hq}/{Hkv} D={D} {dtype}/{cache} page={page}"

    def tokens_of(self, r):
        g = int(np.searchsorted(self.start, r, side="right")) - 1
        if r >= self.start[-1]:
            return None
        L = min(max(0, int(self.prefix[g])), self.table.shape[1] * self.page)
        t = np.arange(L)
        page = self.table[g][t // self.page]
        pre = np.where((page >= 0) & (page < self.k.shape[0]), page * self.page + t % self.page, -1)
        own = self.lists[r][:max(0, min(int(self.lens[r]), self.lists.shape[1]))]
        both = np.concatenate([pre, own]).astype(np.int64)
        return both[(both >= 0) & (both < self.k.shape[0] * self.page)]

    def oracle(self):
        """out, lse and what they may be off by, in float64."""
        kk, vv = (x.double().view(-1, self.Hkv, self.D) for x in (self.k, self.v))
        if self.scales[0] is not None:
            kk, vv = kk * self.scales[0].double()[:, None], vv * self.scales[1].double()[:, None]
        out = torch.zeros((self.R, self.Hq, self.D), dtype=torch.float64)
        lse = torch.full((self.R, self.Hq), -math.inf, dtype=torch.float64)
        off, loff = torch.zeros_like(out), torch.zeros_like(lse)
        per, half = self.Hq // self.Hkv, torch.finfo(self.dtype).eps / 2
        for r in range(self.R):
            tok = self.tokens_of(r)
            if tok is None or not len(tok):
                continue
            k, v = (x[torch.as_tensor(tok)].repeat_interleave(per, 1) for x in (kk, vv))  # [n][Hq][D]
            q = self.q[r].double()
            s = (q * k).sum(-1) * self.scale  # [n][Hq]
            lse[r] = torch.logsumexp(s, 0)
            w = torch.exp(s - lse[r])
            w = torch.where(lse[r].isinf(), 0.0, w)
            out[r] = (w[..., None] * v).sum(0)
            size = (w[..., None] * v.abs()).sum(0)
            # scores: sums of D products in fp32, then a scale and an exponent of a value that large; sums of n
            # weights in fp32, joined a few times; each weight rounded to half a step; the result once more
            reach = ((q * k).abs().sum(-1) * abs(self.scale)).amax(0)
            e = (self.D + 16) * 2.0 ** -24 * reach + (s.abs().amax(0) + 32) * 2.0 ** -23 + (len(tok) + 64) * 2.0 ** -24
            loff[r] = e + lse[r].abs() * 2.0 ** -22
            # (a weight below the type's smallest normal value is off by half of its smallest step)
            tiny = len(tok) * torch.finfo(self.dtype).smallest_normal * 2 * half
            off[r] = half * (out[r].abs() + size) * (1 + 2.0 ** -6) + 2 * e[:, None] * size + tiny * v.abs().amax(0)
        return out, lse, off, loff

    def run(self, dev="cuda", **kw):
        i32 = lambda x: torch.as_tensor(np.ascontiguousarray(x).astype(np.int32)).to(dev)  # noqa: E731
        cache = capi.KVCache(self.k.to(dev), self.v.to(dev), *[None if x is None else x.to(dev) for x in self.scales])
        out = torch.full((self.R, self.Hq, self.D), 7.0, dtype=self.dtype, device=dev)
        lse = torch.full((self.R, self.Hq), 7.0, device=dev)
        args = dict(out=out, lse=lse, scale=self.scale, suffix_slots=i32(self.lists), suffix_len=i32(self.lens))
        args.update(kw)
        return capi.spec_prefix_attention(self.q.to(dev), cache, i32(self.table), i32(self.prefix), i32(self.start), **args)

    def check(self, **kw):
        print("[attention] " + self.name, flush=True)
        got, lse = (x.cpu().double() for x in self.run(**kw))
        out, ref, off, loff = self.oracle()
        if self.pad:
            assert (got[-self.pad:] == 7).all() and (lse[-self.pad:] == 7).all(), "a row behind the last group changed"
            got, lse, out, ref, off, loff = (x[:-self.pad] for x in (got, lse, out, ref, off, loff))
        bad = (got - out).abs() > off
        assert not (bad | got.isnan()).any(), (int(bad.sum()), float(((got - out).abs() - off).max()))
        none = ref.isinf()
        assert torch.equal(none, lse.isinf()) and (lse[none] < 0).all() and (got[none] == 0).all()
        assert ((lse - ref).abs() <= loff)[~none].all(), float(((lse - ref).abs() - loff)[~none].max())
        return got


HEADS = [(1, 1, 64), (8, 1, 128), (8, 8, 64), (32, 8, 128), (6, 2, 80), (12, 4, 96), (40, 2, 128), (16, 2, 256), (3, 1, 8), (5, 5, 200)]


@pytest.mark.parametrize("Hq,Hkv,D", HEADS)
@pytest.mark.parametrize("dtype,cache", [("bf16", None), ("fp16", None), ("bf16", "e4m3"), ("fp16", "e4m3")])
def test_heads_and_types(Hq, Hkv, D, dtype, cache):
    Case([3, 1, 5], [70, 1, 200], [4, 1, 9, 2], Hq, Hkv, D, dtype, cache, page=16, seed=Hq + D).check()


@pytest.mark.parametrize("page", [1, 2, 7, 16, 64, 128, 1000])
@pytest.mark.parametrize("prefix", [[0], [1], [15, 16, 17], [31, 33, 64, 65], [127, 128, 129], [1000, 0, 511, 3]])
def test_lengths_and_pages(page, prefix):
    rows = [(3 * i) % 5 + 1 for i in range(len(prefix))]
    Case(rows, prefix, [1, 0, 5, 33], 8, 2, 64, page=page, seed=page).check()


@pytest.mark.parametrize("rows", [[1], [2] * 9, [17], [64, 1, 33], [200], [0, 4, 0, 0, 7, 0], [1] * 64, [1] * 65, [1, 0, 2] * 150])
def test_rows_per_group(rows):
    Case(rows, [90 + 13 * (i % 7) for i in range(len(rows))], [3, 1, 2], 16, 4, 128, seed=len(rows), pad=3).check()


def test_thousands_of_groups():
    n = 4500
    Case([1] * n, [(7 * i) % 23 for i in range(n)], [1, 0, 2], 2, 1, 64, page=8, seed=21, pad=2).check()


@pytest.mark.parametrize("D,Hq,Hkv", [(128, 8, 1), (64, 16, 2), (128, 6, 1), (120, 8, 1), (256, 8, 1)])
@pytest.mark.parametrize("page", [1, 16, 24, 128])
@pytest.mark.parametrize("prefix", [[1], [31, 32, 33, 95], [96, 97, 127, 200], [2049, 0, 700]])
def test_many_queries(D, Hq, Hkv, page, prefix):
    """Tiles of 128 queries: groups that fill one, two, or just begin another; whole prefixes and holes."""
    rows = [(16, 17, 33, 21)[i % 4] for i in range(len(prefix))]
    c = Case(rows, prefix, [2, 0], Hq, Hkv, D, page=page, seed=page + D, pad=1)
    c.check()
    c.table[0, 0] = -1
    c.table[-1, c.table.shape[1] // 2] = c.k.shape[0]
    flat = [x.view(-1, c.Hkv, c.D) for x in (c.k, c.v)]
    used = torch.zeros(flat[0].shape[0], dtype=torch.bool)
    for r in range(c.R - 1):
        used[torch.as_tensor(c.tokens_of(r))] = True
    for x in flat:
        x[~used] = float("nan")
    c.check()


@pytest.mark.parametrize("suffix", [[1], [16, 17], [32, 33, 31], [0, 300, 1], [64, 65, 640]])
def test_suffixes(suffix):
    Case([4, 2, 6], [40, 0, 129], suffix, 8, 2, 128, seed=len(suffix)).check()


@pytest.mark.parametrize("dtype,cache,Hq,Hkv,D,rows,prefix", [
    ("bf16", None, 32, 8, 128, [1], [9001]), ("bf16", "e4m3", 32, 8, 128, [6, 2], [20011, 300]),
    ("fp16", None, 32, 4, 64, [8] * 5, [3001, 2, 2999, 1500, 700]), ("bf16", None, 16, 1, 256, [40], [5003]),
    ("bf16", None, 8, 2, 128, [100, 3], [2500, 2501])])
def test_long_prefixes(dtype, cache, Hq, Hkv, D, rows, prefix):
    Case(rows, prefix, [7, 1, 3], Hq, Hkv, D, dtype, cache, page=32, seed=D, size=2.0).check()


def test_peaked_scores():
    """Scores far apart, and the largest one first, last, and within the suffix."""
    for where in (0, 700, 1023, -1):
        c = Case([3], [1024], [6], 8, 2, 64, seed=5, size=1.0)
        spot = c.lists[:, 2] if where < 0 else [c.table[0][where // 16] * 16 + where % 16]
        c.k.view(-1, 2, 64)[torch.as_tensor(np.array(spot))] = (c.q[:1, ::4].float() * 12).to(c.dtype)
        c.check()


def test_nothing_to_see_and_holes():
    c = Case([2, 3, 1, 2], [0, 50, 40, 0], [0], 8, 2, 64, seed=1, pad=2)
    c.check()                                    # no prefix, no suffix: zeros
    c = Case([2, 3], [100, 90], [5, 0, 2], 8, 2, 64, seed=2)
    pages = c.k.shape[0]
    c.table[0, 1], c.table[0, 3], c.table[1, 0] = -1, pages, 1 << 30     # pages that are none
    c.lists[0, 0], c.lists[1, 0], c.lists[3, :] = -1, pages * 16, -5      # slots that are none
    c.check()
    c.table[:] = -1                               # a whole prefix of holes
    c.check()
    c = Case([2, 1], [-3, 10 ** 6], [9, -2, 77], 8, 2, 64, seed=3)        # lengths past either end are cut
    c.table[1] = np.arange(c.table.shape[1])
    c.check()


@pytest.mark.parametrize("cache", [None, "e4m3"])
def test_what_lies_outside_does_not_matter(cache):
    """NaN and infinities in unnamed pages, behind a prefix's end and in unnamed slots."""
    c = Case([3, 2], [37, 64], [3, 5], 8, 2, 64, cache=cache, seed=4, spare=3)
    used = torch.zeros(c.k.shape[0] * c.page, dtype=torch.bool)
    for r in range(c.R):
        used[torch.as_tensor(c.tokens_of(r))] = True
    for i, x in enumerate((c.k, c.v)):
        flat = x.view(-1, c.Hkv, c.D)
        if cache:
            flat.view(torch.uint8)[~used] = 0x7F
        else:
            flat[~used] = [float("nan"), float("inf")][i]
            flat[torch.nonzero(~used)[::2, 0]] = [float("-inf"), float("nan")][i]
    c.check()


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
def test_every_value_of_an_8_bit_cache(dtype):
    """One key per row, so that the output is its value: all 256 patterns come through exactly."""
    every = torch.arange(256, dtype=torch.int32).to(torch.uint8).view(torch.float8_e4m3fn)
    for prefix in ([1], [0]):                        # read as a prefix, and from a list
        c = Case([1], prefix, [1 - prefix[0]], 2, 1, 256, dtype, "e4m3", page=4, seed=1)
        c.scales = [torch.ones(1), torch.ones(1)]
        spot = int(c.tokens_of(0)[0])
        c.v.view(-1, 1, 256)[spot, 0] = every
        got = c.run()[0].cpu()[0].float()
        want = every.float().expand(2, 256)
        assert torch.equal(got.isnan(), want.isnan()) and torch.equal(got.nan_to_num(9), want.nan_to_num(9))


def test_infinite_scores():
    c = Case([2], [20], [2], 2, 1, 64, seed=6)
    c.q[:, :, 0] = 1.0
    c.k.view(-1, 1, 64)[torch.as_tensor(c.tokens_of(0)[:10])] = 0
    c.k.view(-1, 1, 64)[torch.as_tensor(c.tokens_of(0)[:10]), :, 0] = float("-inf")
    got = c.check()
    assert torch.isfinite(got).all()
    c.k.view(-1, 1, 64)[:] = 0
    c.k.view(-1, 1, 64)[:, :, 0] = float("-inf")      # every score -inf: zeros
    out, lse = c.run()
    assert (out == 0).all() and (lse == -math.inf).all()
    c.k.view(-1, 1, 64)[torch.as_tensor(c.tokens_of(0)[3]), :, 0] = float("nan")
    out, _ = c.run()
    assert out.isnan().all()                             # a NaN that is seen is not hidden
    c = Case([1], [70], [1], 2, 1, 64, seed=7)          # an infinite value that is seen
    c.v.view(-1, 1, 64)[torch.as_tensor(c.tokens_of(0)[65]), :, 5] = float("inf")
    out, _ = c.run()
    assert (out[:, :, 5] == math.inf).all() and torch.isfinite(out[:, :, 6]).all()


@pytest.mark.parametrize("scale", [0.0, -0.2, 1e-30, 3.0])
def test_factors_of_the_scores(scale):
    c = Case([5], [150], [3, 0], 8, 2, 64, seed=12, size=0.5)
    c.scale = scale
    c.check()
    c = Case([5], [150], [3, 0], 8, 2, 64, cache="e4m3", seed=13, size=0.5)
    c.scale = scale
    c.scales = [torch.tensor([-0.7, 0.0]), torch.tensor([-1.3, 0.5])]  # turned round, and nothing at all
    c.check()


def test_a_nan_stays_in_its_row():
    """A query of NaN, and one that sees a NaN of its own, next to others in the same tile."""
    c = Case([6, 3], [90, 70], [4, 2, 3], 8, 2, 64, seed=14)
    ref, lref = (x.cpu() for x in c.run())
    c.q[2, 3] = float("nan")
    c.k.view(-1, 2, 64)[int(c.lists[7, 0])] = float("nan")
    got, lse = (x.cpu() for x in c.run())
    bad = torch.zeros(c.R, c.Hq, dtype=torch.bool)
    bad[2, 3], bad[7] = True, True
    assert got[bad].isnan().all() and lse[bad].isnan().all()
    assert torch.equal(got[~bad], ref[~bad]) and torch.equal(lse[~bad], lref[~bad])


def test_named_streams():
    """The stream argument, as an object and as a handle, while the current stream is another."""
    c = Case([9, 3], [700, 90], [5, 2], 16, 4, 128, seed=15)
    ref = c.run()
    torch.cuda.synchronize()
    for _ in range(3):
        s = torch.cuda.Stream()
        for stream in (s, s.cuda_stream):
            got = c.run(stream=stream, workspace=None)
            junk = torch.full((1 << 22,), float("nan"), device="cuda")  # takes memory given away too early
            s.synchronize()
            assert all(torch.equal(a, b) for a, b in zip(got, ref))
            del junk


def test_strides_and_layouts():
    c = Case([3, 2], [50, 33], [4, 2], 8, 2, 64, seed=8)
    ref, lref = c.run()
    i32 = lambda x: torch.as_tensor(np.ascontiguousarray(x).astype(np.int32)).cuda()  # noqa: E731
    wide = torch.zeros((c.Hq, c.R, 3, 64), dtype=c.dtype, device="cuda")
    q = wide.permute(1, 0, 2, 3)[:, :, 1]
    q.copy_(c.q)
    both = torch.zeros((c.k.shape[0], 2, c.Hkv, c.page, 64), dtype=c.dtype, device="cuda")
    kc, vc = both[:, 0].transpose(1, 2), both[:, 1].transpose(1, 2)
    kc.copy_(c.k)
    vc.copy_(c.v)
    out = torch.zeros((c.R, c.Hq + 1, 64), dtype=c.dtype, device="cuda")[:, 1:]
    got, _ = capi.spec_prefix_attention(q, capi.KVCache(kc, vc), i32(c.table), i32(c.prefix), i32(c.start),
                                        suffix_slots=i32(c.lists), suffix_len=i32(c.lens), out=out)
    assert torch.equal(got, ref)
    none, _ = capi.spec_prefix_attention(q, capi.KVCache(kc, vc), i32(c.table), i32(c.prefix), i32(c.start))
    c.lens[:] = 0
    want, _ = c.run()
    assert torch.equal(none, want)
    c2 = Case([5], [0], [4, 2], 8, 2, 64, seed=9)         # no page table at all
    got, _ = capi.spec_prefix_attention(c2.q.cuda(), capi.KVCache(c2.k.cuda(), c2.v.cuda()), None, None, i32(c2.start),
                                        suffix_slots=i32(c2.lists), suffix_len=i32(c2.lens))
    assert torch.equal(got, c2.run()[0])


def test_long_cache_offsets():
    """Pages and slots that lie more than 2^32 elements into the cache."""
    Hkv, D, page = 8, 128, 64
    pages = (1 << 32) // (page * Hkv * D) + 4
    k = torch.zeros((pages, page, Hkv, D), dtype=torch.bfloat16, device="cuda")
    v = torch.zeros_like(k)
    c = Case([3], [200], [2], 16, Hkv, D, page=page, seed=10)
    n = c.k.shape[0]
    k[-n:], v[-n:] = c.k.cuda(), c.v.cuda()
    ref, _ = c.run()
    i32 = lambda x: torch.as_tensor(np.ascontiguousarray(x).astype(np.int32)).cuda()  # noqa: E731
    got, _ = capi.spec_prefix_attention(c.q.cuda(), capi.KVCache(k, v), i32(c.table + pages - n), i32(c.prefix), i32(c.start),
                                        suffix_slots=i32(c.lists + (pages - n) * page), suffix_len=i32(c.lens))
    assert torch.equal(got, ref)


def test_same_bits_every_time_on_streams_and_in_graphs():
    c = Case([9, 3, 20], [700, 90, 1300], [5, 2, 8], 16, 4, 128, seed=11)
    dev = "cuda"
    i32 = lambda x: torch.as_tensor(np.ascontiguousarray(x).astype(np.int32)).to(dev)  # noqa: E731
    q, cache = c.q.cuda(), capi.KVCache(c.k.cuda(), c.v.cuda())
    table, lens, start, lists, sl = i32(c.table), i32(c.prefix), i32(c.start), i32(c.lists), i32(c.lens)
    call = lambda: capi.spec_prefix_attention(q, cache, table, lens, start, suffix_slots=lists, suffix_len=sl, want_lse=True)  # noqa: E731
    ref = [x.clone() for x in call()]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    for _ in range(3):
        got = []
        for s in streams:
            with torch.cuda.stream(s):
                got.append(call())
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for x in got for a, b in zip(x, ref))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = call()
    for i in range(4):
        q.normal_()
        lens.copy_(i32(c.prefix - 37 * i).clamp(min=0))
        graph.replay()
        torch.cuda.synchronize()
        now = call()
        assert all(torch.equal(a, b) for a, b in zip(held, now))
