"""Argument checks and host helpers of the steps on either side of the verification (no GPU)."""
import ctypes
import math
import re

import numpy as np
import pytest
import torch

from lossless_speculative_sampling_amd import capi

FAKE = ctypes.c_void_p(0x1000)
OFF = ctypes.c_void_p(0x1001)


def _probs(**kw):
    a = dict(draft=FAKE, target=FAKE, dtype=0, B=2, K=3, V=10000, tokens=FAKE, u=FAKE, v=FAKE, ut=0, flags=0, k=FAKE, t=FAKE,
             ws=FAKE, n=1 << 20)
    a.update(kw)
    return capi.load().cdll.spec_verify_probs(a["draft"], 300, 100, a["target"], 400, 100, a["dtype"], a["B"], a["K"], a["V"],
                                              a["tokens"], None, a["u"], a["v"], a["ut"], a["flags"], a["k"], a["t"], None,
                                              None, None, a["ws"], a["n"], None)


@pytest.mark.parametrize("bad,rc", [
    (dict(draft=None), -1), (dict(target=None), -1), (dict(tokens=None), -1), (dict(u=None), -1), (dict(v=None), -1),
    (dict(k=None), -1), (dict(t=None), -1), (dict(B=0), -1), (dict(K=0), -1), (dict(V=0), -1), (dict(flags=1), -1),
    (dict(flags=10), -1), (dict(dtype=3), -2), (dict(dtype=9), -2), (dict(ut=1), -2), (dict(target=OFF), -1),
    (dict(draft=OFF), -1), (dict(u=OFF), -1), (dict(B=1 << 30), -1), (dict(B=1 << 30, V=100), -1), (dict(ws=None), -3), (dict(n=10), -3), (dict(ws=OFF), -3)])
def test_verify_probs_errors(bad, rc):
    assert _probs(**bad) == rc


def test_verify_probs_workspace():
    f = capi.spec_verify_probs_workspace_bytes
    assert f(0, 10) == 0 and f(1, 0) == 0 and f(1 << 30, 1 << 30) == 0
    assert f(1, 1) == f(512, 8192) == 0 and 0 < f(1, 8193) <= f(16, 128256) <= f(512, 151936)
    assert f(1, (1 << 31) - 1) == 0 and 0 < f(1, 0x7fff0000) < 1 << 20


def _cache(**kw):
    a = dict(k=0x1000, v=0x1000, dtype=1, num_pages=4, page_size=16, heads=2, head_dim=64, page_stride=2048, token_stride=128,
             head_stride=64, k_scale=None, v_scale=None)
    a.update(kw)
    return capi._Cache(*a.values())


def _append(cache=None, **kw):
    a = dict(q=FAKE, qo=FAKE, k=FAKE, v=FAKE, dtype=1, T=3, Hq=4, H=2, D=64, pos=FAKE, slots=FAKE, freqs=FAKE, rot=64,
             scale=1.0, flags=0, qs=256, qos=256)
    a.update(kw)
    c = _cache() if cache is None else cache
    return capi.load().cdll.spec_kv_append(a["q"], a["qs"], 64, a["qo"], a["qos"], 64, a["k"], 128, 64, a["v"], 128, 64,
                                           a["dtype"], a["T"], a["Hq"], a["H"], a["D"], a["pos"], a["slots"], a["freqs"],
                                           a["rot"], a["scale"], a["flags"], ctypes.byref(c) if c else None, None, None)


@pytest.mark.parametrize("bad,rc", [
    (dict(q=None, k=None), -1), (dict(qo=None), -1), (dict(v=None), -1), (dict(slots=None), -1), (dict(T=-1), -1),
    (dict(T=1 << 24), -1), (dict(D=0), -1), (dict(D=2000), -1), (dict(Hq=0), -1), (dict(H=0), -1), (dict(H=3), -1),
    (dict(rot=3), -1), (dict(rot=66), -1), (dict(rot=-2), -1), (dict(pos=None), -1), (dict(freqs=None), -1),
    (dict(flags=2), -1), (dict(scale=math.inf), -1), (dict(scale=math.nan), -1), (dict(dtype=0), -2), (dict(dtype=3), -2),
    (dict(dtype=2), -2), (dict(q=OFF), -1), (dict(k=OFF), -1), (dict(qs=512), -1), (dict(T=0), 0)])
def test_append_errors(bad, rc):
    assert _append(**bad) == rc


@pytest.mark.parametrize("bad,rc", [
    (dict(k=None), -1), (dict(num_pages=0), -1), (dict(page_size=0), -1), (dict(heads=1), -1), (dict(head_dim=32), -1),
    (dict(num_pages=1 << 30), -1), (dict(dtype=0), -2), (dict(dtype=2), -2), (dict(v=0x1001), -1)])
def test_append_cache_errors(bad, rc):
    assert _append(cache=_cache(**bad)) == rc


def _attend(cache=None, **kw):
    a = dict(q=FAKE, dtype=1, R=3, Hq=4, G=2, start=FAKE, table=FAKE, pages=2, lens=FAKE, lists=FAKE, S=3, sl=FAKE, scale=0.1,
             out=ctypes.c_void_p(0x2000), ws=FAKE, n=1 << 40, qs=256)
    a.update(kw)
    c = _cache() if cache is None else cache
    return capi.load().cdll.spec_prefix_attention(a["q"], a["qs"], 64, a["dtype"], a["R"], a["Hq"], ctypes.byref(c), a["G"],
                                                  a["start"], a["table"], a["pages"], a["lens"], a["lists"], a["S"], a["sl"],
                                                  a["scale"], a["out"], 256, 64, None, a["ws"], a["n"], None)


@pytest.mark.parametrize("bad,rc", [
    (dict(q=None), -1), (dict(out=None), -1), (dict(out=FAKE), -1), (dict(start=None), -1), (dict(table=None), -1),
    (dict(lens=None), -1), (dict(lists=None), -1), (dict(sl=None), -1), (dict(pages=-1), -1), (dict(S=-1), -1),
    (dict(R=-1), -1), (dict(G=0), -1), (dict(Hq=3), -1), (dict(Hq=0), -1), (dict(scale=math.nan), -1), (dict(dtype=0), -2),
    (dict(dtype=2), -2), (dict(q=OFF), -1), (dict(out=ctypes.c_void_p(0x2008)), -1), (dict(qs=260), -1), (dict(ws=None), -3),
    (dict(n=0), -3), (dict(ws=OFF), -3), (dict(R=0), 0), (dict(pages=1 << 28), -1)])
def test_attention_errors(bad, rc):
    assert _attend(**bad) == rc


@pytest.mark.parametrize("bad,rc", [
    (dict(head_dim=60), -1), (dict(head_dim=264), -1), (dict(token_stride=130), -1), (dict(page_stride=1), -1), (dict(k=0x1008), -1),
    (dict(v=0x1002), -1), (dict(dtype=3, k=0x1004), -1), (dict(page_stride=-2048), -1), (dict(head_stride=-64), -1), (dict(heads=3), -1), (dict(dtype=4), -2)])
def test_attention_cache_errors(bad, rc):
    assert _attend(cache=_cache(**bad)) == rc


def test_attention_workspace():
    f = capi.spec_prefix_attention_workspace_bytes
    assert f(8, 2, 8, 2, 128, 4096, 5) > f(8, 2, 8, 2, 128, 4096, 0) > 0 and f(0, 1, 8, 8, 8, 0, 0) > 0
    for bad in ((-1, 1, 8, 8, 64, 10, 0), (4, 0, 8, 8, 64, 10, 0), (4, 1, 8, 3, 64, 10, 0), (4, 1, 8, 0, 64, 10, 0),
                (4, 1, 8, 8, 257, 10, 0), (4, 1, 8, 8, 12, 10, 0), (4, 1, 8, 8, 64, -1, 0), (4, 1, 8, 8, 64, 1 << 31, 0),
                (4, 1, 8, 8, 64, 10, -1), (1 << 30, 1, 8, 8, 64, 10, 0), (4, 1 << 30, 8, 8, 64, 10, 0)):
        assert f(*bad) == 0


def test_tree_rows_errors():
    L = capi.load().cdll

    def rc(B=2, N=5, depth=3, hole=None):
        p = [FAKE] * 8
        if hole is not None:
            p[hole] = None
        return L.spec_tree_rows(*p[:4], B, N, depth, *p[4:], None)

    assert all(rc(hole=i) == -1 for i in range(8))
    assert rc(B=0) == rc(N=0) == rc(depth=0) == rc(B=1 << 24) == -1


@pytest.mark.parametrize("rot,base,factor,low,high,orig", [(128, 10000.0, 1.0, 1.0, 4.0, 8192), (64, 500000.0, 8.0, 1.0, 4.0, 8192),
                                                           (2, 10.0, 2.0, 1.0, 32.0, 100), (96, 1e6, 32.0, 2.0, 2.0, 4096)])
def test_rope_frequencies(rot, base, factor, low, high, orig):
    f = base ** (-np.arange(0, rot, 2) / rot)
    n = orig * f / (2 * math.pi)
    g = (n >= low).astype(float) if low == high else np.clip((n - low) / (high - low), 0, 1)
    np.testing.assert_allclose(capi.spec_rope_frequencies(rot, base, factor, low, high, orig), f * (g + (1 - g) / factor), rtol=1e-14)


def test_rope_frequencies_stretch_all_and_errors():
    plain = np.array(capi.spec_rope_frequencies(16, 10000.0))
    all_ = np.array(capi.spec_rope_frequencies(16, 10000.0, 4.0, math.inf, math.inf))
    np.testing.assert_allclose(all_, plain / 4, rtol=1e-15)
    np.testing.assert_allclose(capi.spec_rope_frequencies(16, 10000.0, 4.0, 1.0, math.inf), plain / 4, rtol=1e-15)
    for bad in (dict(rot_dim=0), dict(rot_dim=3), dict(rot_dim=2048), dict(base=0.0), dict(base=math.inf), dict(factor=0.5),
                dict(low=3.0, high=2.0), dict(low=math.nan), dict(low=-math.inf), dict(original_len=0), dict(factor=math.nan)):
        with pytest.raises(capi.SpecError):
            capi.spec_rope_frequencies(**{"rot_dim": 8, **bad})


def _t(*shape, dtype=torch.int32):
    return torch.zeros(shape, dtype=dtype)


BF = torch.bfloat16


@pytest.mark.parametrize("change,msg", [
    (dict(target=_t(2, 4, 10, dtype=torch.float64)), "target must be"), (dict(target=_t(2, 1, 10, dtype=BF)), "no drafted position"),
    (dict(draft=_t(2, 3, 10, dtype=torch.float16)), "same dtype"), (dict(draft=_t(2, 3, 11, dtype=BF)), "draft must be"),
    (dict(draft=None), "are required"), (dict(tokens=_t(2, 3, dtype=torch.int64)), "tokens must be"),
    (dict(tokens=_t(3, 2).T), "contiguous"), (dict(accept_u=_t(2, 3, dtype=BF)), "accept_u must be"),
    (dict(sample_v=_t(2, dtype=torch.float64)), "sample_v must be"), (dict(sample_v=_t(3, dtype=torch.float32)), "sample_v must have"),
    (dict(draft_lens=_t(3)), "draft_lens must have"), (dict(target=_t(2, 10, 4, dtype=BF).transpose(1, 2)), "last dimension"),
    (dict(workspace=_t(8)), "workspace"), (dict(), "device tensor expected")])
def test_verify_probs_binding(change, msg):
    a = dict(draft=_t(2, 3, 10, dtype=BF), target=_t(2, 4, 10, dtype=BF), tokens=_t(2, 3), accept_u=_t(2, 3, dtype=torch.float32),
             sample_v=_t(2, dtype=torch.float32))
    with pytest.raises(ValueError, match=re.escape(msg)):
        capi.spec_verify_probs(**{**a, **change})


def _kv(dtype=BF, heads=2, D=16):
    return capi.KVCache(_t(3, 4, heads, D, dtype=dtype), _t(3, 4, heads, D, dtype=dtype))


@pytest.mark.parametrize("change,msg", [
    (dict(k=None), "come together"), (dict(cache=None), "come together"), (dict(slots=None), "come together"),
    (dict(v=_t(5, 2, 8, dtype=BF)), "same shape"), (dict(q=_t(4, 4, 16, dtype=BF)), "k must be"),
    (dict(q=_t(5, 4, 16, dtype=torch.float16)), "same dtype"), (dict(slots=_t(4)), "slots must have"),
    (dict(cache=_kv(heads=3)), "do not match"), (dict(cache=_kv(torch.float32)), "unsupported dtype"),
    (dict(cache=capi.KVCache(_t(3, 4, 2, 16, dtype=BF), _t(3, 2, 4, 16, dtype=BF).transpose(1, 2))), "same strides"),
    (dict(cache=capi.KVCache(_t(3, 4, 2, 16, dtype=BF), _t(3, 4, 2, 16, dtype=BF), _t(2, dtype=torch.float32))), "8-bit"),
    (dict(rotary=capi.Rotary(_t(9, dtype=torch.float64))), "at most 8"), (dict(rotary=capi.Rotary(_t(8, dtype=torch.float32))), "must be torch.float64"),
    (dict(positions=None, rotary=capi.Rotary(_t(8, dtype=torch.float64))), "positions is required"),
    (dict(q_out=_t(5, 4, 8, dtype=BF)), "like q"), (dict(status=_t(4)), "status must have"), (dict(), "device tensor expected")])
def test_append_binding(change, msg):
    a = dict(k=_t(5, 2, 16, dtype=BF), v=_t(5, 2, 16, dtype=BF), positions=_t(5), slots=_t(5), cache=_kv(), q=_t(5, 4, 16, dtype=BF))
    with pytest.raises(ValueError, match=re.escape(msg)):
        capi.spec_kv_append(**{**a, **change})


@pytest.mark.parametrize("change,msg", [
    (dict(q=_t(5, 4, 16, dtype=torch.float32)), "bf16 or fp16"), (dict(q=_t(5, 3, 16, dtype=BF)), "do not serve"),
    (dict(row_start=_t(1)), "row_start"), (dict(page_table=_t(3, 2)), "page_table must have"), (dict(prefix_len=None), "prefix_len is required"),
    (dict(suffix_len=None), "suffix_len is required"), (dict(suffix_slots=_t(4, 3)), "suffix_slots must have"),
    (dict(out=_t(5, 4, 8, dtype=BF)), "like q"), (dict(lse=_t(5, 4)), "lse must be"), (dict(workspace=_t(1)), "workspace"),
    (dict(), "device tensor expected")])
def test_attention_binding(change, msg):
    a = dict(q=_t(5, 4, 16, dtype=BF), cache=_kv(), page_table=_t(2, 3), prefix_len=_t(2), row_start=_t(3), suffix_slots=_t(5, 3),
             suffix_len=_t(5))
    with pytest.raises(ValueError, match=re.escape(msg)):
        capi.spec_prefix_attention(**{**a, **change})


def test_tree_rows_binding():
    for change, msg in ((dict(tokens=_t(4)), "[B][N]"), (dict(parents=_t(2, 3)), "parents must have"), (dict(ctx_len=_t(3)), "ctx_len must have"),
                        (dict(max_depth=0), "max_depth"), (dict(slots=_t(2, 4, dtype=torch.int64)), "slots must be"), (dict(), "device tensor")):
        a = dict(tokens=_t(2, 4), parents=_t(2, 4), slots=_t(2, 4), ctx_len=_t(2), max_depth=3)
        with pytest.raises(ValueError, match=re.escape(msg)):
            capi.spec_tree_rows(**{**a, **change})
