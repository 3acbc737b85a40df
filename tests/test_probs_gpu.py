"""spec_verify_probs against its definition in 64 bits on the host (needs an MI355X)."""
import numpy as np
import pytest
import torch

from lossless_speculative_sampling_amd import capi

pytestmark = pytest.mark.gpu
DT = {"fp32": torch.float32, "bf16": torch.bfloat16, "fp16": torch.float16}


def oracle(p, q, tokens, u, v, lens, kind="rows"):
    """p [B][K][V] or None, q [B][K+1][V], all float64 numpy: k, t*, emitted, residual mass, status."""
    B, K1, V = q.shape
    K = K1 - 1
    out = dict(k=np.zeros(B, int), t=np.full(B, -1), emitted=np.full((B, K1), -1), mass=np.zeros(B), status=np.zeros(B, int))

    def draft(b, j):
        if kind == "uniform":
            return np.full(V, 1.0 / V)
        if kind == "point":
            x = np.zeros(V)
            x[tokens[b, j]] = 1.0
            return x
        return p[b, j]

    for b in range(B):
        L = K if lens is None else int(lens[b])
        if not 0 <= L <= K:
            out["status"][b] = capi.ST_BAD_PARAM
            continue
        k, bad = 0, 0
        while k < L:
            s = tokens[b, k]
            if not 0 <= s < V:
                bad = capi.ST_BAD_TOKEN
                break
            ps, qs = draft(b, k)[s], q[b, k, s]
            if not (np.isfinite(ps) and np.isfinite(qs) and ps >= 0 and qs >= 0):
                bad = capi.ST_BAD_PROB
                break
            if not 0 <= u[b, k] <= 1:
                bad = capi.ST_BAD_PARAM
                break
            if ps == 0:
                out["status"][b] |= capi.ST_OUTSIDE_DRAFT_SUPPORT
            if not u[b, k] * ps < qs:
                break
            k += 1
        if bad:
            out["status"][b] |= bad
            continue
        rows = [q[b, k]] + ([draft(b, k)] if k < L else [])
        if not 0 <= v[b] <= 1:
            out["status"][b] |= capi.ST_BAD_PARAM
            continue
        if any(not np.isfinite(r).all() or (r < 0).any() for r in rows):
            out["status"][b] |= capi.ST_BAD_PROB
            continue
        w = np.maximum(rows[0] - rows[1], 0) if k < L else rows[0]
        if w.sum() == 0 and k < L and rows[0].sum() > 0:
            out["status"][b] |= capi.ST_EMPTY_RESIDUAL
            w = rows[0]
        elif k < L:
            out["mass"][b] = w.sum()
        if w.sum() == 0:
            out["status"][b] |= capi.ST_BAD_PROB
            continue
        c = np.cumsum(w)
        hit = np.nonzero(c > v[b] * c[-1])[0]
        t = hit[0] if len(hit) else np.nonzero(w > 0)[0][-1]
        out["k"][b], out["t"][b] = k, t
        out["emitted"][b, :k], out["emitted"][b, k] = tokens[b, :k], t
    return out


def rows_of(rng, B, K, V, sharp=1.0, noise=0.7, cut=1e-6):
    z = rng.standard_normal((B, K + 1, V)) * sharp - 1.1 * np.log1p(rng.permutation(V))

    def soft(x):
        e = np.exp(x - x.max(-1, keepdims=True))
        e /= e.sum(-1, keepdims=True)
        e[e < cut] = 0
        return e / e.sum(-1, keepdims=True)

    return soft(z[:, :K] + noise * rng.standard_normal((B, K, V))), soft(z)


def check(p, q, tokens, u, v, lens=None, flags=0, kind="rows", **kw):
    """p and q device tensors (any strides); compares every output."""
    K = q.shape[1] - 1
    dev = lambda x: None if x is None else torch.as_tensor(x).cuda()  # noqa: E731
    tok = torch.as_tensor(np.asarray(tokens, np.int32)).cuda()
    ln = None if lens is None else torch.as_tensor(np.asarray(lens, np.int32)).cuda()
    r = capi.spec_verify_probs(p, q, tok, dev(u), dev(v), draft_lens=ln, flags=flags, **kw)
    ref = oracle(None if p is None else p.double().cpu().numpy(), q.double().cpu().numpy(), np.asarray(tokens),
                 np.asarray(u, np.float64), np.asarray(v, np.float64), lens, kind)
    np.testing.assert_array_equal(r.status.cpu().numpy(), ref["status"])
    np.testing.assert_array_equal(r.k.cpu().numpy(), ref["k"])
    np.testing.assert_array_equal(r.tstar.cpu().numpy(), ref["t"])
    np.testing.assert_array_equal(r.emitted.cpu().numpy(), ref["emitted"])
    # fp64 sums rounded once to fp32: half a step, and the sums' own order
    np.testing.assert_allclose(r.resid_mass.cpu().numpy(), ref["mass"], rtol=2.0 ** -24 + 1e-12, atol=1e-44)
    assert K + 1 == r.emitted.shape[1]
    return r, ref


@pytest.mark.parametrize("dtype", ["fp32", "bf16", "fp16"])
@pytest.mark.parametrize("B,K,V", [(1, 1, 1), (2, 1, 2), (3, 4, 7), (5, 3, 1000), (2, 5, 2048), (3, 2, 2049), (7, 63, 513),
                                   (2, 70, 300), (4, 3, 8192), (3, 3, 8193), (2, 2, 40001), (40, 2, 131073)])
def test_against_the_definition(dtype, B, K, V):
    rng = np.random.default_rng(B * 1000 + K * 100 + V)
    p, q = rows_of(rng, B, K, V)
    tokens = np.stack([[rng.choice(V, p=p[b, j]) for j in range(K)] for b in range(B)])
    pd, qd = (torch.as_tensor(x).to(DT[dtype]).cuda() for x in (p, q))
    u, v = rng.random((B, K)), rng.random(B)
    if dtype == "fp32":
        u, v = u.astype(np.float32), v.astype(np.float32)
    print(f"[probs] {dtype} B={B} K={K} V={V}", flush=True)
    check(pd, qd, tokens, u, v)
    check(pd, qd, tokens, u, v, lens=rng.integers(0, K + 1, B))
    check(None, qd, tokens, u, v, flags=capi.SPEC_UNIFORM_DRAFT, kind="uniform")
    check(None, qd, tokens, u, v, flags=capi.SPEC_POINT_DRAFT, kind="point", lens=rng.integers(0, K + 1, B))


@pytest.mark.parametrize("V", [37, 20000])
def test_strided_and_unaligned_rows(V):
    rng = np.random.default_rng(V)
    B, K = 4, 3
    p, q = rows_of(rng, B, K, V)
    tokens = rng.integers(0, V, (B, K))
    wide = torch.zeros((K + 1, B, V + 13), dtype=torch.bfloat16, device="cuda")
    qd = wide.transpose(0, 1)[:, :, 3:3 + V]
    qd.copy_(torch.as_tensor(q))
    wide2 = torch.zeros((B, K, 2, V), dtype=torch.bfloat16, device="cuda")
    pd = wide2[:, :, 1]
    pd.copy_(torch.as_tensor(p))
    check(pd, qd, tokens, rng.random((B, K)), rng.random(B))
    one = torch.as_tensor(p[:1, :1]).to(torch.bfloat16).cuda().expand(B, K, V)  # one row for all
    check(one, qd, tokens, rng.random((B, K)), rng.random(B))


def test_a_row_longer_than_the_cells_of_one_tile():
    """2.2 million tokens: cells of two tiles each."""
    V = 2200003
    g = torch.Generator().manual_seed(1)
    q, p = (torch.rand((3, n, V), generator=g).cuda() ** 4 for n in (2, 1))
    check(p, q, np.array([[5], [V - 1], [1 << 20]]), np.array([[1.0], [0.0], [1.0]]), np.array([0.25, 0.999999, 0.5]), lens=[1, 1, 1])


@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
def test_more_rows_than_the_caches_hold(dtype):
    rng = np.random.default_rng(8)
    B, V = (300, 131073) if dtype == "fp32" else (600, 131073)
    p, q = rows_of(rng, 2, 2, V)
    at = np.arange(B) % 2
    pd, qd = (torch.as_tensor(x).to(DT[dtype]).cuda()[at] for x in (p, q))
    tok = rng.integers(0, 99, (B, 2)).astype(np.int32)
    u, v = rng.random((B, 2)), rng.random(B)
    r = capi.spec_verify_probs(pd, qd, torch.as_tensor(tok).cuda(), torch.as_tensor(u).cuda(), torch.as_tensor(v).cuda())
    some = np.concatenate([np.arange(8), np.arange(B - 8, B)])
    ref = oracle(pd[some].double().cpu().numpy(), qd[some].double().cpu().numpy(), tok[some], u[some], v[some], None)
    for name, key in (("k", "k"), ("tstar", "t"), ("emitted", "emitted"), ("status", "status")):
        np.testing.assert_array_equal(getattr(r, name).cpu().numpy()[some], ref[key])


def test_edges_of_the_random_numbers():
    q = torch.tensor([[[0.0, 0.25, 0.0, 0.75, 0.0], [0.0, 0.5, 0.5, 0.0, 0.0]]]).cuda().expand(6, 2, 5).contiguous()
    p = torch.tensor([[[0.0, 1.0, 0.0, 0.0, 0.0]]]).cuda().expand(6, 1, 5).contiguous()
    tok = np.ones((6, 1), int)
    # u = q/p exactly is a rejection; just below accepts; v = 0 takes the first token with mass, v = 1 the last
    u = np.array([[0.25], [0.2499999], [0.0], [1.0], [0.25], [0.1]])
    v = np.array([0.0, 0.0, 1.0, 1.0, 0.5, 0.5])
    r, ref = check(p, q, tok, u, v)
    assert ref["k"].tolist() == [0, 1, 1, 0, 0, 1]
    # v * total on a running mass exactly: it has to exceed it
    assert ref["t"].tolist() == [3, 1, 2, 3, 3, 2]


def test_rows_where_nothing_is_left_and_bad_input():
    B, V = 12, 9000
    q = torch.full((B, 2, V), 1.0 / V, device="cuda")
    p = q[:, :1].clone()
    tok = np.full((B, 1), 5)
    u, v = np.full((B, 1), 1.0), np.full(B, 0.5)
    lens = np.ones(B, int)
    q[1, 0, 5] = float("nan")           # the drafted token's own probability
    q[2, 0, 8999] = float("inf")        # in the row the draw sums
    q[3, 0, 100] = -1e-3
    p[4, 0, 8000] = float("nan")
    tok[5] = V
    tok[6] = -1
    u[7] = float("nan")
    v[8] = 1.5
    lens[9] = 2
    q[10] = 0.0                         # a target row without mass
    lens[10] = 0
    lens[11] = -1
    r, ref = check(p, q, tok, u, v, lens=lens)
    assert ref["status"][0] == capi.ST_EMPTY_RESIDUAL  # p == q, u = 1: rejected with nothing left
    assert (ref["status"][1:5] == capi.ST_BAD_PROB).all() and (ref["status"][5:7] == capi.ST_BAD_TOKEN).all()
    assert (ref["status"][[7, 8, 9, 11]] == capi.ST_BAD_PARAM).all() and ref["status"][10] == capi.ST_BAD_PROB
    # a bad value behind the scan's end does not matter
    q2 = torch.full((1, 3, 50), 0.02, device="cuda")
    p2 = torch.full((1, 2, 50), 0.02, device="cuda")
    p2[0, 0, 3] = 1.0
    q2[0, 2], p2[0, 1, 3], = float("nan"), float("nan")
    check(p2, q2, np.array([[3, 77]]), np.array([[0.9, 7.0]]), np.array([0.3]))


def test_many_requests():
    rng = np.random.default_rng(9)
    p, q = rows_of(rng, 1, 2, 6)
    B = 70000
    pd, qd = (torch.as_tensor(x).float().cuda().expand(B, -1, -1) for x in (p, q))
    tok = rng.integers(0, 6, (B, 2)).astype(np.int32)
    u, v = rng.random((B, 2)), rng.random(B)
    r = capi.spec_verify_probs(pd, qd, torch.as_tensor(tok).cuda(), torch.as_tensor(u).cuda(), torch.as_tensor(v).cuda())
    some = np.concatenate([np.arange(200), np.arange(B - 200, B)])
    ref = oracle(pd[:400].double().cpu().numpy(), qd[:400].double().cpu().numpy(), tok[some], u[some], v[some], None)
    for name, key in (("k", "k"), ("tstar", "t"), ("emitted", "emitted"), ("status", "status")):
        np.testing.assert_array_equal(getattr(r, name).cpu().numpy()[some], ref[key])


def test_outputs_given_and_a_named_stream():
    rng = np.random.default_rng(4)
    p, q = rows_of(rng, 5, 3, 20000)
    pd, qd = (torch.as_tensor(x).float().cuda() for x in (p, q))
    tok = torch.as_tensor(rng.integers(0, 9, (5, 3)).astype(np.int32)).cuda()
    u, v = torch.rand((5, 3), device="cuda"), torch.rand(5, device="cuda")
    ref = capi.spec_verify_probs(pd, qd, tok, u, v)
    i32 = lambda *n: torch.full(n, -9, dtype=torch.int32, device="cuda")  # noqa: E731
    out = capi.ProbsOut(i32(5), i32(5), i32(5, 4), torch.full((5,), -9.0, device="cuda"), i32(5))
    ws = torch.full((capi.spec_verify_probs_workspace_bytes(5, 20000),), 0xAB, dtype=torch.uint8, device="cuda")  # not cleared
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    for stream in (s, s.cuda_stream):
        got = capi.spec_verify_probs(pd, qd, tok, u, v, workspace=ws, out=out, stream=stream)
        alone = capi.spec_verify_probs(pd, qd, tok, u, v, stream=stream)
        s.synchronize()
        assert got is out
        for name in ("k", "tstar", "emitted", "resid_mass", "status"):
            assert torch.equal(getattr(out, name), getattr(ref, name)) and torch.equal(getattr(alone, name), getattr(ref, name))


def test_outside_the_drafts_support():
    q = torch.tensor([[[0.5, 0.5, 0.0], [0.2, 0.3, 0.5]]] * 2).cuda()
    p = torch.tensor([[[1.0, 0.0, 0.0]]] * 2).cuda()
    r, ref = check(p, q, np.array([[1], [2]]), np.array([[0.9], [0.0]]), np.array([0.1, 0.7]))
    assert ref["status"].tolist() == [capi.ST_OUTSIDE_DRAFT_SUPPORT] * 2 and ref["k"].tolist() == [1, 0]


def test_agrees_with_spec_verify_on_its_own_uniforms():
    """The same outcome as spec_verify where the processed distributions and random numbers are its own."""
    import oracle as lib
    from lossless_speculative_sampling_amd import synth
    w = synth.vanilla(B=64, K=4, V=1024)
    prm = capi.params_tensor(w.temperature, w.top_k, w.top_p)
    d, t = torch.from_numpy(w.draft).cuda(), torch.from_numpy(w.target).cuda()
    tok = torch.zeros((w.B, w.K), dtype=torch.int32, device="cuda")
    r = capi.spec_verify(d, t, w.K, prm, tok, seed=w.seed, flags=capi.SPEC_SAMPLE_DRAFT)
    ref = lib.verify(w.draft, w.target, lib.FP32, w.K, w.params(), tokens=tok.cpu().numpy(), seed=w.seed, round_=0)
    fine = torch.from_numpy(ref.flags == 0)
    U = lib.uniforms(w.seed, 0, w.B, w.K)
    u, v = np.ascontiguousarray(U[:, :w.K, 0]), U[np.arange(w.B), r.k.cpu().numpy(), 1]
    got = capi.spec_verify_probs(torch.softmax(d.double(), -1).float()[:, :w.K].contiguous(), torch.softmax(t.double(), -1).float(),
                                 tok, torch.from_numpy(u).cuda(), torch.from_numpy(v).cuda())
    assert fine.sum() > 32
    assert torch.equal(got.k.cpu()[fine], r.k.cpu()[fine]) and torch.equal(got.tstar.cpu()[fine], r.tstar.cpu()[fine])


def test_streams_and_graph_replays():
    rng = np.random.default_rng(3)
    B, K, V = 6, 4, 50000
    p, q = rows_of(rng, B, K, V)
    pd, qd = (torch.as_tensor(x).float().cuda() for x in (p, q))
    tok = torch.as_tensor(rng.integers(0, 40, (B, K)).astype(np.int32)).cuda()
    u, v = torch.rand((B, K), device="cuda"), torch.rand(B, device="cuda")
    ref = capi.spec_verify_probs(pd, qd, tok, u, v)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    for _ in range(3):
        got = []
        for s in streams:
            with torch.cuda.stream(s):
                got.append(capi.spec_verify_probs(pd, qd, tok, u, v))
        torch.cuda.synchronize()
        for g in got:
            assert torch.equal(g.tstar, ref.tstar) and torch.equal(g.emitted, ref.emitted)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = capi.spec_verify_probs(pd, qd, tok, u, v)
    for i in range(4):
        u.uniform_()
        v.uniform_()
        graph.replay()
        torch.cuda.synchronize()
        now = capi.spec_verify_probs(pd, qd, tok, u, v)
        assert torch.equal(held.k, now.k) and torch.equal(held.tstar, now.tstar) and torch.equal(held.resid_mass, now.resid_mass)
