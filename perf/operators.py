"""What the operators of a speculative round around the verification are measured on.

Four operators: verification of drafted tokens from given probabilities and random numbers
("verify"), the rows of draft trees ("tree"), rotary positions with the append of keys and values
to a paged cache ("append"), and attention of rows that share a long prefix ("attention").

`own` false: the operators in plain torch operations, 32 bits (64 where a sum over the vocabulary
or the angle of a far position needs them), rounded once at the end.  `own` true: the package's
operators on the same state.
"""
import math

import numpy as np
import torch

own = False

DEV = "cuda"
TYPES = {"fp32": torch.float32, "fp64": torch.float64, "bf16": torch.bfloat16, "fp16": torch.float16,
         "e4m3": torch.float8_e4m3fn}
BYTES = {"fp32": 4, "fp64": 8, "bf16": 2, "fp16": 2, "e4m3": 1}
E4M3_MOST = 448.0


# ---- the cases -----------------------------------------------------------------------------

def listed():
    return [
        # one request with a small vocabulary: all latency
        dict(name="verify_one", op="verify", B=1, K=4, V=1024, dtype="fp32", uniform="fp32", draft="rows", ragged=False),
        # the benchmark's batch and vocabulary, processed probabilities in 32 bits, ragged draft lengths
        dict(name="verify_batch", op="verify", B=16, K=5, V=128256, dtype="fp32", uniform="fp64", draft="rows", ragged=True),
        # the branch tree's 512 chains of seven tokens, probabilities kept in bf16
        dict(name="verify_chains", op="verify", B=512, K=7, V=151936, dtype="bf16", uniform="fp32", draft="rows", ragged=False),
        # 16 requests, the drafted chain of five tokens and 32 guessed outcomes hanging off it
        dict(name="tree_outcomes", op="tree", B=16, N=37, depth=6),
        # 512 draft trees of 255 nodes
        dict(name="tree_wide", op="tree", B=512, N=255, depth=12),
        # one token for each of 16 requests, the whole head rotated
        dict(name="append_step", op="append", T=16, Hq=32, Hkv=8, D=128, rot=128, interleaved=False, dtype="bf16",
             cache="bf16", page=16, far=4096, run=False),
        # all branches' tokens of a round, half of the head rotated pairwise, an 8-bit cache
        dict(name="append_branches", op="append", T=592, Hq=32, Hkv=8, D=128, rot=64, interleaved=True, dtype="bf16",
             cache="e4m3", page=32, far=131072, run=False),
        # a prompt of odd length at far positions of a scaled context
        dict(name="append_prompt", op="append", T=16383, Hq=32, Hkv=8, D=128, rot=128, interleaved=False, dtype="bf16",
             cache="bf16", page=64, far=1000000, run=True),
        # one request, one token, a context of ordinary length
        dict(name="attend_one", op="attention", G=1, rows=1, ragged=False, Hq=32, Hkv=8, D=128, dtype="bf16",
             cache="bf16", page=16, prefix=1000, suffix=1, lse=False),
        # 64 requests with eight branches each, ragged contexts, small heads in fp16
        dict(name="attend_trees", op="attention", G=64, rows=8, ragged=True, Hq=32, Hkv=4, D=64, dtype="fp16",
             cache="fp16", page=32, prefix=2049, suffix=8, lse=True),
        # 16 requests, a drafted chain and 32 guessed outcomes with their rollouts, long contexts
        dict(name="attend_outcomes", op="attention", G=16, rows=37, ragged=True, Hq=32, Hkv=8, D=128, dtype="bf16",
             cache="bf16", page=64, prefix=8192, suffix=11, lse=False),
        # one request's chain of six tokens scored over a very long context held in 8 bits
        dict(name="attend_long", op="attention", G=1, rows=6, ragged=False, Hq=32, Hkv=8, D=128, dtype="bf16",
             cache="e4m3", page=128, prefix=131071, suffix=6, lse=False),
    ]


def _spread(rng, low, high):
    """A whole number of [low, high], even over its logarithm."""
    return max(low, min(high, int(round(math.exp(rng.uniform(math.log(low), math.log(high + 0.49)))))))


def draw(rng):
    op = rng.choice(["verify", "tree", "append", "append", "attention", "attention"])
    if op == "verify":
        V, K = _spread(rng, 500, 200000), rng.randint(1, 12)
        return dict(op=op, B=_spread(rng, 1, max(1, min(512, 300000000 // (V * (K + 1))))), K=K, V=V,
                    dtype=rng.choice(["fp32", "bf16", "fp16"]), uniform=rng.choice(["fp32", "fp64"]),
                    draft=rng.choice(["rows", "rows", "point", "uniform"]), ragged=rng.random() < 0.5)
    if op == "tree":
        return dict(op=op, B=_spread(rng, 1, 512), N=_spread(rng, 1, 250), depth=rng.randint(1, 16))
    if op == "append":
        D, Hkv = rng.choice([64, 80, 96, 128, 256]), rng.choice([1, 2, 4, 8])
        dtype = rng.choice(["bf16", "fp16"])
        return dict(op=op, T=_spread(rng, 1, 16000 * 8 * 128 // (Hkv * D * 4)), Hq=Hkv * rng.choice([1, 3, 4, 8]), Hkv=Hkv,
                    D=D, rot=rng.choice([D, D, D // 2]), interleaved=rng.random() < 0.5, dtype=dtype,
                    cache=rng.choice([dtype, dtype, "e4m3"]), page=rng.choice([1, 16, 32, 64, 128]),
                    far=_spread(rng, 100, 1000000), run=rng.random() < 0.5)
    D, Hkv, G = rng.choice([64, 80, 128, 128, 256]), rng.choice([1, 2, 4, 8]), _spread(rng, 1, 64)
    rows, Hq, dtype = _spread(rng, 1, 40), Hkv * rng.choice([1, 3, 4, 8]), rng.choice(["bf16", "fp16"])
    most = min(4000000000 // (G * rows * Hq * D), 60000000 // (G * Hkv * D), 131072)
    return dict(op=op, G=G, rows=rows, ragged=rng.random() < 0.7, Hq=Hq, Hkv=Hkv, D=D, dtype=dtype,
                cache=rng.choice([dtype, dtype, "e4m3"]), page=rng.choice([1, 16, 32, 64, 128]),
                prefix=_spread(rng, 20, max(20, most)), suffix=rng.randint(1, 14), lse=rng.random() < 0.5)


# ---- verification from given probabilities ---------------------------------------------------

def _prepare_verify(c, g, rng):
    B, K, V = c["B"], c["K"], c["V"]
    dtype = TYPES[c["dtype"]]
    base = -1.1 * torch.log1p(torch.randperm(V, device=DEV, generator=g).float())

    def rows(x):  # processed rows: tokens with next to no probability are cut off
        p = torch.softmax(x, -1)
        p = torch.where(p > 1e-7, p, 0.0)
        return (p / p.sum(-1, keepdim=True))

    z = torch.randn((B, K + 1, V), device=DEV, generator=g) + base
    target = rows(z).to(dtype)
    draft = None
    if c["draft"] == "rows":
        p = rows(z[:, :K] + 0.8 * torch.randn((B, K, V), device=DEV, generator=g))
        tokens = torch.multinomial(p.reshape(B * K, V), 1, generator=g).reshape(B, K)
        draft = p.to(dtype)
    elif c["draft"] == "point":
        tokens = torch.multinomial(target[:, :K].float().reshape(B * K, V), 1, generator=g).reshape(B, K)
    else:
        tokens = torch.randint(0, V, (B, K), device=DEV, generator=g)
    lens = torch.randint(0, K + 1, (B,), device=DEV, generator=g, dtype=torch.int32) if c["ragged"] else None
    u = TYPES[c["uniform"]]
    return dict(draft=draft, target=target, tokens=tokens.to(torch.int32), lens=lens,
                u=torch.rand((B, K), device=DEV, generator=g, dtype=u), v=torch.rand(B, device=DEV, generator=g, dtype=u))


def _run_verify(s):
    c = s["case"]
    if own:
        from lossless_speculative_sampling_amd import capi
        flags = {"rows": 0, "point": capi.SPEC_POINT_DRAFT, "uniform": capi.SPEC_UNIFORM_DRAFT}[c["draft"]]
        r = capi.spec_verify_probs(s["draft"], s["target"], s["tokens"], s["u"], s["v"], draft_lens=s["lens"], flags=flags)
        return {"k": r.k, "tstar": r.tstar, "emitted": r.emitted, "resid_mass": r.resid_mass}
    target, tokens = s["target"], s["tokens"].long()
    B, K, V = target.shape[0], tokens.shape[1], target.shape[2]
    at = torch.arange(B, device=DEV)
    j = torch.arange(K + 1, device=DEV)
    lens = torch.full((B,), K, device=DEV) if s["lens"] is None else s["lens"].long()
    qs = target[:, :K].gather(2, tokens[..., None])[..., 0].double()
    if c["draft"] == "rows":
        ps = s["draft"].gather(2, tokens[..., None])[..., 0].double()
    else:
        ps = torch.full_like(qs, 1.0 if c["draft"] == "point" else 1.0 / V)
    accept = (s["u"].double() * ps < qs) & (j[:K] < lens[:, None])
    k = accept.long().cumprod(1).sum(1)
    rejected = k < lens
    qk = target[at, k].double()
    last = k.clamp(max=K - 1)
    if c["draft"] == "rows":
        pk = s["draft"][at, last].double()
    elif c["draft"] == "point":
        pk = (torch.arange(V, device=DEV) == tokens[at, last][:, None]).double()
    else:
        pk = torch.full_like(qk, 1.0 / V)
    w = torch.where(rejected[:, None], (qk - pk).clamp(min=0.0), qk)
    mass = w.sum(1)
    w = torch.where((rejected & (mass <= 0))[:, None], qk, w)
    run_ = w.cumsum(1)
    tstar = (run_ <= (s["v"].double() * run_[:, -1])[:, None]).sum(1)
    emitted = torch.where(j < k[:, None], torch.nn.functional.pad(tokens, (0, 1)), torch.where(j == k[:, None], tstar[:, None], -1))
    return {"k": k.int(), "tstar": tstar.int(), "emitted": emitted.int(),
            "resid_mass": torch.where(rejected, mass, 0.0).float()}


def _exact_verify(c, s):
    """The residual mass alone has a value in 64 bits; the tokens are whole numbers."""
    B, K, V = c["B"], c["K"], c["V"]
    lens = [K] * B if s["lens"] is None else s["lens"].tolist()
    tokens, u = s["tokens"].tolist(), s["u"].double().tolist()
    mass = []
    for b in range(B):
        said = 0.0
        for j in range(lens[b]):
            q = s["target"][b, j].double()
            t = tokens[b][j]
            if c["draft"] == "rows":
                p = s["draft"][b, j].double()
            elif c["draft"] == "point":
                p = torch.zeros_like(q)
                p[t] = 1.0
            else:
                p = torch.full_like(q, 1.0 / V)
            if not u[b][j] * p[t].item() < q[t].item():
                said = (q - torch.minimum(p, q)).sum().item()
                break
        mass.append(said)
    return {"k": None, "tstar": None, "emitted": None, "resid_mass": torch.tensor(mass, dtype=torch.float64)}


def _work_verify(c):
    B, K, V, e = c["B"], c["K"], c["V"], BYTES[c["dtype"]]
    rows = 2 if c["draft"] == "rows" else 1  # of each request the scan ends in one row of either side
    small = B * (K * (4 + BYTES[c["uniform"]]) + BYTES[c["uniform"]] + 4 * (K + 1) + 12)
    return {"bytes": B * V * e * rows + 2 * B * K * e + small, "flops": 3 * B * V}


# ---- the rows of draft trees -----------------------------------------------------------------

def _prepare_tree(c, g, rng):
    B, N = c["B"], c["N"]
    parents, depth = np.full((B, N), -1, np.int32), np.ones((B, N), np.int32)
    for n in range(1, N):  # parents stand before their children; a chain first, then forks off it
        p = np.where(rng.random(B) < 0.3, n - 1, rng.integers(-1, n, B))
        deep = np.where(p >= 0, depth[np.arange(B), p], 0)
        p = np.where(deep >= c["depth"] + 1, -1, p)  # a few nodes are one deeper than the rows hold
        parents[:, n], depth[:, n] = p, np.where(p >= 0, depth[np.arange(B), p], 0) + 1
    tokens = rng.integers(0, 128256, (B, N)).astype(np.int32)
    tokens[rng.random((B, N)) < 0.02] = -1
    tokens[np.arange(N)[None, :] >= rng.integers(max(1, 3 * N // 4), N + 1, B)[:, None]] = -1  # padded at the end
    slots = rng.permutation(2 * B * N)[:B * N].reshape(B, N).astype(np.int32)
    ctx = rng.integers(0, 8192, B).astype(np.int32)
    return {k: torch.from_numpy(v).to(DEV) for k, v in dict(tokens=tokens, parents=parents, slots=slots, ctx=ctx).items()}


def _run_tree(s):
    depth = s["case"]["depth"]
    if own:
        from lossless_speculative_sampling_amd import capi
        r = capi.spec_tree_rows(s["tokens"], s["parents"], s["slots"], s["ctx"], depth)
        return {"positions": r.positions, "append": r.append_slots, "slots": r.suffix_slots, "len": r.suffix_len}
    tokens, parents, slots = s["tokens"], s["parents"].long(), s["slots"]
    B, N = tokens.shape
    n = torch.arange(N, device=DEV)
    bad = (tokens < 0) | (parents < -1) | (parents >= n)
    up = (n == torch.where(bad, -1, parents)[..., None]).float()  # [B][N][N]: row n marks its parent
    reach = torch.linalg.matrix_power(up + torch.eye(N, device=DEV), 1 << depth.bit_length()) > 0.5
    deep = reach.sum(2)
    fine = (deep <= depth) & ~(reach & bad[:, None, :]).any(2)
    at = torch.where(reach & fine[..., None], (deep - 1)[:, None, :], depth)
    lists = torch.full((B, N, depth + 1), -1, dtype=torch.int32, device=DEV)
    lists.scatter_(2, at, slots[:, None, :].expand(B, N, N))
    return {"positions": torch.where(fine, s["ctx"][:, None] + deep - 1, -1).int(), "append": torch.where(fine, slots, -1),
            "slots": lists[..., :depth].contiguous(), "len": torch.where(fine, deep, 0).int()}


def _work_tree(c):
    return {"bytes": c["B"] * c["N"] * 4 * (3 + 3 + c["depth"]) + 4 * c["B"], "flops": c["B"] * c["N"] * c["depth"]}


# ---- rotary positions and the append to a paged cache ----------------------------------------

def _frequencies(rot, base=500000.0, factor=8.0, low=1.0, high=4.0, original=8192):
    """Inverse frequencies with the slow ones stretched for a long context."""
    f = base ** (-np.arange(0, rot, 2, dtype=np.float64) / rot)
    keep = np.clip((original * f / (2 * np.pi) - low) / (high - low), 0.0, 1.0)
    return f * (keep + (1.0 - keep) / factor)


def _prepare_append(c, g, rng):
    T, Hq, Hkv, D, dtype = c["T"], c["Hq"], c["Hkv"], c["D"], TYPES[c["dtype"]]
    pages = 2 * -(-T // c["page"])
    some = lambda *shape: torch.randn(shape, device=DEV, generator=g)  # noqa: E731

    def cache():
        x = some(pages, c["page"], Hkv, D)
        return x.to(TYPES[c["cache"]])

    if c["run"]:  # a prompt: neighbouring positions, whole pages in any order
        positions = c["far"] + np.arange(T)
        slots = (rng.permutation(pages)[:, None] * c["page"] + np.arange(c["page"])).reshape(-1)[:T]
    else:  # tokens of many requests and branches
        positions = rng.integers(0, c["far"], T)
        slots = rng.permutation(pages * c["page"])[:T]
    scales = (0.5 + torch.rand((2, Hkv), device=DEV, generator=g)) / 32 if c["cache"] == "e4m3" else [None, None]
    return dict(q=some(T, Hq, D).to(dtype), k=some(T, Hkv, D).to(dtype), v=some(T, Hkv, D).to(dtype), kc=cache(), vc=cache(),
                positions=torch.from_numpy(positions.astype(np.int32)).to(DEV), slots=torch.from_numpy(slots.astype(np.int32)).to(DEV),
                freqs=torch.from_numpy(_frequencies(c["rot"])).to(DEV), stretch=1.0 + 0.1 * math.log(8.0), ks=scales[0], vs=scales[1])


def _rotate(x, cos, sin, rot, interleaved):
    x = x.float()
    y, rest = x[..., :rot], x[..., rot:]
    a, b = (y[..., 0::2], y[..., 1::2]) if interleaved else (y[..., :rot // 2], y[..., rot // 2:])
    r, i = a * cos - b * sin, b * cos + a * sin
    return torch.cat([torch.stack([r, i], -1).flatten(-2) if interleaved else torch.cat([r, i], -1), rest], -1)


def _store(cache, slots, x, scale):
    if scale is None:
        cache.view(-1, *cache.shape[2:])[slots] = x.to(cache.dtype)
    else:
        x = (x / scale[:, None]).clamp(-E4M3_MOST, E4M3_MOST).to(cache.dtype)
        cache.view(torch.uint8).view(-1, *cache.shape[2:])[slots] = x.view(torch.uint8)


def _run_append(s):
    c = s["case"]
    if own:
        from lossless_speculative_sampling_amd import capi
        cache = capi.KVCache(s["kc"], s["vc"], s["ks"], s["vs"])
        rotary = capi.Rotary(s["freqs"], interleaved=c["interleaved"], scale=s["stretch"])
        q = capi.spec_kv_append(s["k"], s["v"], s["positions"], s["slots"], cache, rotary, q=s["q"])
        return {"q": q, "k": s["kc"], "v": s["vc"]}
    angle = s["positions"].double()[:, None] * s["freqs"]
    cos, sin = ((f(angle) * s["stretch"]).float()[:, None, :] for f in (torch.cos, torch.sin))
    slots = s["slots"].long()
    q = _rotate(s["q"], cos, sin, c["rot"], c["interleaved"]).to(s["q"].dtype)
    _store(s["kc"], slots, _rotate(s["k"], cos, sin, c["rot"], c["interleaved"]), s["ks"])
    _store(s["vc"], slots, s["v"].float(), s["vs"])
    return {"q": q, "k": s["kc"], "v": s["vc"]}


def _exact_append(c, s):
    half = c["rot"] // 2
    turn = torch.polar(torch.full((c["T"], 1, half), s["stretch"], dtype=torch.float64, device=DEV),
                       (s["positions"].double()[:, None] * s["freqs"])[:, None])

    def rotated(x):
        x = x.double()
        y = x.clone()
        first, second = (slice(0, c["rot"], 2), slice(1, c["rot"], 2)) if c["interleaved"] else (slice(0, half), slice(half, c["rot"]))
        z = torch.complex(x[..., first], x[..., second]) * turn
        y[..., first], y[..., second] = z.real, z.imag
        return y

    def held(cache, x, scale):
        y = cache.to(torch.float64).view(-1, c["Hkv"], c["D"])
        y[s["slots"].long()] = x if scale is None else (x / scale.double()[:, None]).clamp(-E4M3_MOST, E4M3_MOST)
        return y.view(cache.shape)

    return {"q": rotated(s["q"]), "k": held(s["kc"], rotated(s["k"]), s["ks"]), "v": held(s["vc"], s["v"].double(), s["vs"])}


def _work_append(c):
    e, o, T = BYTES[c["dtype"]], BYTES[c["cache"]], c["T"]
    return {"bytes": T * c["D"] * (2 * c["Hq"] * e + 2 * c["Hkv"] * (e + o)) + 8 * T + 4 * c["rot"],
            "flops": T * (c["Hq"] + c["Hkv"]) * c["rot"] * 3}


# ---- attention of rows that share a long prefix ----------------------------------------------

def _prepare_attention(c, g, rng):
    G, Hq, Hkv, D, page, S = c["G"], c["Hq"], c["Hkv"], c["D"], c["page"], c["suffix"]
    rows = np.linspace(max(1, c["rows"] // 2), c["rows"], G).round().astype(int) if c["ragged"] else np.full(G, c["rows"])
    rows = rng.permutation(rows)  # as many in all for every seed
    R = int(rows.sum())
    lens = rng.integers(max(1, c["prefix"] // 2), c["prefix"] + 1, G) if c["ragged"] else np.full(G, c["prefix"])
    wide = -(-c["prefix"] // page)
    behind = -(-(G * S + R * S) // page)  # pages of the tokens behind the prefixes
    pages = rng.permutation(G * wide + behind)
    slots = (pages[G * wide:, None] * page + np.arange(page)).reshape(-1)
    slots = slots[rng.permutation(slots.size)]
    group = np.repeat(np.arange(G), rows)
    # a row sees a part of its group's drafted chain, then its own tokens
    chain, mine = slots[:G * S].reshape(G, S), slots[G * S:G * S + R * S].reshape(R, S)
    shared = rng.integers(0, S, R)
    lists = np.where(np.arange(S) < shared[:, None], chain[group], mine)
    suffix_len = rng.integers(shared + 1, S + 1)
    start = np.concatenate([[0], np.cumsum(rows)])
    whole = lambda x: torch.from_numpy(np.ascontiguousarray(x).astype(np.int32)).to(DEV)  # noqa: E731
    kv = [torch.randn((pages.size, page, Hkv, D), device=DEV, generator=g).to(TYPES[c["cache"]]) for _ in range(2)]
    scales = 0.5 + torch.rand((2, Hkv), device=DEV, generator=g) if c["cache"] == "e4m3" else [None, None]
    return dict(q=torch.randn((R, Hq, D), device=DEV, generator=g).to(TYPES[c["dtype"]]), kc=kv[0], vc=kv[1], ks=scales[0], vs=scales[1],
                table=whole(pages[:G * wide].reshape(G, wide)), lens=whole(lens), start=whole(start), lists=whole(lists),
                suffix_len=whole(suffix_len), most=int(rows.max()))


def _taken(cache, slots, scale):
    """The cache's rows at `slots`, in 32 bits."""
    raw = cache.view(torch.uint8) if cache.dtype == TYPES["e4m3"] else cache
    x = raw.view(-1, *cache.shape[2:])[slots].view(cache.dtype).float()
    return x if scale is None else x * scale[:, None]


def _run_attention(s):
    c = s["case"]
    if own:
        from lossless_speculative_sampling_amd import capi
        cache = capi.KVCache(s["kc"], s["vc"], s["ks"], s["vs"])
        out, lse = capi.spec_prefix_attention(s["q"], cache, s["table"], s["lens"], s["start"], suffix_slots=s["lists"],
                                              suffix_len=s["suffix_len"], want_lse=c["lse"])
        return {"out": out, "lse": lse}
    q, start, lists = s["q"], s["start"].long(), s["lists"].long()
    G, n, page, per = c["G"], s["most"], c["page"], c["Hq"] // c["Hkv"]
    R, (Hq, Hkv, D), S = q.shape[0], (c["Hq"], c["Hkv"], c["D"]), c["suffix"]
    row = torch.arange(R, device=DEV)
    group = torch.searchsorted(start[1:].contiguous(), row, right=True)
    local = row - start[group]
    at = (start[:-1, None] + torch.arange(n, device=DEV)).clamp(max=R - 1)  # [G][n], padded groups
    spots = (s["table"].long()[..., None] * page + torch.arange(page, device=DEV)).flatten(1)
    k, v = _taken(s["kc"], spots, s["ks"]), _taken(s["vc"], spots, s["vs"])  # [G][L][Hkv][D]
    L = spots.shape[1]
    x = q.float()[at].view(G, n, Hkv, per, D).transpose(1, 2) / math.sqrt(D)  # [G][Hkv][n][per][D]
    far = (x.reshape(G, Hkv, n * per, D) @ k.permute(0, 2, 3, 1)).view(G, Hkv, n, per, L)
    far = far.masked_fill(torch.arange(L, device=DEV) >= s["lens"][:, None, None, None, None], -math.inf)
    ks, vs = _taken(s["kc"], lists[at], s["ks"]), _taken(s["vc"], lists[at], s["vs"])  # [G][n][S][Hkv][D]
    near = x @ ks.permute(0, 3, 1, 4, 2)  # [G][Hkv][n][per][S]
    near = near.masked_fill(torch.arange(S, device=DEV) >= s["suffix_len"][at][:, None, :, None, None], -math.inf)
    top = torch.maximum(far.amax(-1), near.amax(-1))[..., None]
    far, near = torch.exp(far - top), torch.exp(near - top)
    total = far.sum(-1, keepdim=True) + near.sum(-1, keepdim=True)
    y = (far.view(G, Hkv, n * per, L) @ v.transpose(1, 2)).view(G, Hkv, n, per, D) + near @ vs.permute(0, 3, 1, 2, 4)
    out = (y / total).transpose(1, 2).reshape(G, n, Hq, D)[group, local].to(q.dtype)
    lse = (top + total.log())[..., 0].transpose(1, 2).reshape(G, n, Hq)[group, local] if c["lse"] else None
    return {"out": out, "lse": lse}


def _exact_attention(c, s):
    Hkv, D, per = c["Hkv"], c["D"], c["Hq"] // c["Hkv"]
    flat = [x.view(-1, Hkv, D) if x.dtype != TYPES["e4m3"] else x.view(torch.uint8).view(-1, Hkv, D) for x in (s["kc"], s["vc"])]
    factor = [1.0 if x is None else x.double()[:, None] for x in (s["ks"], s["vs"])]
    rows_of = lambda i, slots: flat[i][slots].view(s["kc"].dtype).double() * factor[i]  # noqa: E731
    out, lse = [], []
    start, lens, suffix = s["start"].tolist(), s["lens"].tolist(), s["suffix_len"].tolist()
    for g in range(c["G"]):
        t = torch.arange(lens[g], device=DEV)
        spots = s["table"][g].long()[t // c["page"]] * c["page"] + t % c["page"]
        k, v = rows_of(0, spots).transpose(0, 1).contiguous(), rows_of(1, spots).transpose(0, 1).contiguous()  # [Hkv][L][D]
        kt = k.transpose(1, 2).contiguous()
        for r in range(start[g], start[g + 1]):
            x = s["q"][r].double().view(Hkv, per, D)
            own_ = s["lists"][r, :suffix[r]].long()
            kn, vn = rows_of(0, own_).transpose(0, 1).contiguous(), rows_of(1, own_).transpose(0, 1).contiguous()
            score = torch.cat([x @ kt, x @ kn.transpose(1, 2).contiguous()], -1) * D ** -0.5
            norm = torch.logsumexp(score, -1, keepdim=True)
            w = torch.exp(score - norm)
            out.append((w[..., :lens[g]] @ v + w[..., lens[g]:] @ vn).reshape(-1, D))
            lse.append(norm.reshape(-1))
    return {"out": torch.stack(out), "lse": torch.stack(lse) if c["lse"] else None}


def _work_attention(c):
    mean = lambda n: n * 0.75 if c["ragged"] else n  # noqa: E731
    R, L, e = c["G"] * mean(c["rows"]), mean(c["prefix"]), BYTES[c["dtype"]]
    behind = c["G"] * c["suffix"] / 2 + R * c["suffix"] / 2  # tokens behind the prefixes, each read once
    return {"bytes": 2 * (c["G"] * L + behind) * c["Hkv"] * c["D"] * BYTES[c["cache"]] + 2 * R * c["Hq"] * c["D"] * e,
            "flops": 4.0 * R * (L + 0.75 * c["suffix"]) * c["Hq"] * c["D"]}


# ---- what the tools call -----------------------------------------------------------------------

def prepare(case, seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(int(seed))
    make = {"verify": _prepare_verify, "tree": _prepare_tree, "append": _prepare_append, "attention": _prepare_attention}
    return dict(make[case["op"]](case, g, np.random.default_rng(int(seed))), case=case)


def run(state):
    return {"verify": _run_verify, "tree": _run_tree, "append": _run_append, "attention": _run_attention}[state["case"]["op"]](state)


def exact(case, seed):
    if case["op"] == "tree":
        return None
    state = prepare(case, seed)
    return {"verify": _exact_verify, "append": _exact_append, "attention": _exact_attention}[case["op"]](case, state)


def work(case):
    return {"verify": _work_verify, "tree": _work_tree, "append": _work_append, "attention": _work_attention}[case["op"]](case)
