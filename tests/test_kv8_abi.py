"""Rotary positions and the 8-bit cache on the host: the C ABI's refusals (every case here fails validation, or
stops at the device check, before any launch), workspace sizes, frequencies, and the oracles themselves."""

import math
import os
import re

import numpy as np
import pytest
import torch

import oracle.kv8 as ok8
import oracle.rotary as orot
import sparse_attention_lightning_bf16_amd as lx
from sparse_attention_lightning_bf16_amd import _lib

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
NULL, SHAPE, UNSUP, DEVICE = -1, -2, -3, -4
P = 1 << 20          # a fake, 256-byte aligned address: never dereferenced


def test_every_declared_function_is_bound():
    for header in ("lix_rotary.h", "lix_kv8.h"):
        src = re.sub(r"/\*.*?\*/", "", open(os.path.join(ROOT, "include", header)).read(), flags=re.S)
        for name in re.findall(r"\b(lix_[a-z0-9_]+)\s*\(", src):
            assert name in _lib.SIGNATURES and hasattr(lx.load(), name), name


def rotary_call(x=P, xs=(64, 64, 64), pos=P, ps=(1, 1), f=P, N0=2, N1=2, H=2, D=64, rot=32, start=0, layout=0, scale=1.0,
                inverse=0, dtype=0, out=P, os_=(64, 64, 64)):
    return lx.load().lix_rotary(x, *xs, pos, *ps, f, N0, N1, H, D, rot, start, layout, scale, inverse, dtype, out, *os_,
                                None)


@pytest.mark.parametrize("kw,code", [
    (dict(x=None), NULL), (dict(pos=None), NULL), (dict(f=None), NULL), (dict(out=None), NULL),
    (dict(N0=0), SHAPE), (dict(N1=-1), SHAPE), (dict(H=0), SHAPE), (dict(D=0), SHAPE), (dict(rot=0), SHAPE),
    (dict(rot=3), SHAPE), (dict(rot=66), SHAPE), (dict(start=-1), SHAPE), (dict(start=33), SHAPE),
    (dict(start=2147483647), SHAPE), (dict(layout=2), SHAPE), (dict(dtype=3), SHAPE), (dict(xs=(-1, 0, 0)), SHAPE),
    (dict(os_=(0, 0, -64)), SHAPE), (dict(ps=(0, -1)), SHAPE),
    (dict(D=1026, rot=2), UNSUP), (dict(x=P + 1), UNSUP), (dict(out=P + 2, dtype=2), UNSUP), (dict(f=P + 4), UNSUP),
    (dict(pos=P + 2), UNSUP), (dict(N0=1 << 16, N1=1 << 15), UNSUP), (dict(xs=(1 << 41, 0, 0)), UNSUP),
    (dict(), DEVICE), (dict(x=P + 2, start=32), DEVICE), (dict(ps=(0, 0)), DEVICE),
])
def test_rotary_validation(kw, code):
    assert rotary_call(**kw) == code


CACHE = dict(kp=P, vp=P, ks=P, vs=P, np_=8, page=64, table=P, mp=4, lens=P)


def append_call(k=P, s=(512, 128, 64), v=P, dtype=0, B=2, S=4, H=2, D=64, new=None, **kw):
    c = dict(CACHE, **kw)
    return lx.load().lix_kv8_append(k, *s, v, *s, dtype, B, S, H, D, c["kp"], c["vp"], c["ks"], c["vs"], c["np_"],
                                    c["page"], c["table"], c["mp"], c["lens"], new, None)


COMMON = [
    (dict(kp=None), NULL), (dict(ks=None), NULL), (dict(table=None), NULL), (dict(lens=None), NULL),
    (dict(B=0), SHAPE), (dict(S=0), SHAPE), (dict(H=0), SHAPE), (dict(D=0), SHAPE), (dict(np_=0), SHAPE),
    (dict(mp=0), SHAPE), (dict(page=-16), SHAPE), (dict(dtype=2), SHAPE), (dict(s=(-8, 128, 64)), SHAPE),
    (dict(page=8), UNSUP), (dict(page=48), UNSUP), (dict(page=256), UNSUP), (dict(D=96), UNSUP), (dict(D=512), UNSUP),
    (dict(np_=1 << 26), UNSUP),                       # 2^31 token rows
    (dict(mp=1 << 24), UNSUP), (dict(s=(512, 128, 68)), UNSUP), (dict(s=(1 << 41, 128, 64)), UNSUP),
    (dict(kp=P + 8), UNSUP), (dict(ks=P + 2), UNSUP), (dict(table=P + 1), UNSUP), (dict(lens=P + 2), UNSUP),
    (dict(), DEVICE),
]


@pytest.mark.parametrize("kw,code", COMMON + [
    (dict(k=None), NULL), (dict(v=None), NULL), (dict(vp=None), NULL), (dict(k=P + 8), UNSUP), (dict(new=P + 1), UNSUP),
    (dict(S=(1 << 30) + 1), UNSUP), (dict(B=1, s=(-8, 128, 64)), DEVICE),     # one row: its stride reaches nothing
])
def test_append_validation(kw, code):
    assert append_call(**kw) == code


def attention_call(q=P, s=(512, 256, 64), dtype=0, B=2, S=1, Hq=4, H=2, D=64, start=None, qlens=None, ratio=1,
                   scale=0.125, idx=None, topk=0, out=P, lse=P, ws=P, ws_bytes=1 << 30, **kw):
    c = dict(CACHE, **kw)
    return lx.load().lix_kv8_attention(q, *s, dtype, B, S, Hq, H, D, c["kp"], c["vp"], c["ks"], c["vs"], c["np_"],
                                       c["page"], c["table"], c["mp"], c["lens"], start, qlens, ratio, scale, idx, topk,
                                       out, lse, ws, ws_bytes, None)


QUERY = [
    (dict(q=None), NULL), (dict(lse=None), NULL), (dict(Hq=3), SHAPE), (dict(Hq=0), SHAPE), (dict(ratio=0), SHAPE),
    (dict(scale=-1.0), SHAPE), (dict(scale=math.nan), SHAPE), (dict(scale=math.inf), SHAPE), (dict(q=P + 8), UNSUP),
    (dict(lse=P + 2), UNSUP), (dict(start=P + 2), UNSUP), (dict(qlens=P + 1), UNSUP),
    (dict(S=1 << 29, Hq=4), UNSUP),
]


@pytest.mark.parametrize("kw,code", [c for c in COMMON if "s" not in c[0]] + QUERY + [
    (dict(s=(-8, 256, 64)), SHAPE), (dict(s=(512, 256, 68)), UNSUP), (dict(vp=None), NULL), (dict(out=None), NULL),
    (dict(idx=P, topk=0), SHAPE), (dict(idx=P + 2, topk=4), UNSUP), (dict(out=P + 8), UNSUP), (dict(mp=64, ws=None), NULL),
    (dict(ws=P + 16), UNSUP), (dict(mp=64, ws_bytes=16), SHAPE), (dict(mp=64), DEVICE),
    (dict(ws=None, ws_bytes=0), DEVICE),             # one part: no workspace
])
def test_attention_validation(kw, code):
    assert attention_call(**kw) == code


def weights_call(q=P, s=(512, 256, 64), dtype=0, B=2, S=1, Hq=4, H=2, D=64, start=None, qlens=None, ratio=1,
                 scale=0.125, lse=P, w=P, width=256, acc=0, ws=None, ws_bytes=0, **kw):
    c = dict(CACHE, **kw)
    return lx.load().lix_kv8_token_weights(q, *s, dtype, B, S, Hq, H, D, c["kp"], c["ks"], c["np_"], c["page"], c["table"],
                                           c["mp"], c["lens"], start, qlens, ratio, scale, lse, w, width, acc, ws, ws_bytes, None)


@pytest.mark.parametrize("kw,code", QUERY + [
    (dict(w=None), NULL), (dict(width=255), SHAPE), (dict(w=P + 2), UNSUP), (dict(page=20), UNSUP), (dict(ws=P + 8), UNSUP),
    (dict(S=512), NULL), (dict(S=512, ws=P), SHAPE), (dict(S=512, ws=P, ws_bytes=1 << 20), DEVICE), (dict(D=32), UNSUP),
    (dict(), DEVICE),
])
def test_token_weights_validation(kw, code):
    assert weights_call(**kw) == code


def evict_call(B=2, H=2, D=64, w=P, width=256, new=P, nmp=2, keep=100, recent=10, sinks=4, nl=P, kept=P, nw=P, ws=P,
               ws_bytes=1 << 30, **kw):
    c = dict(CACHE, **kw)
    return lx.load().lix_kv8_evict(c["kp"], c["vp"], c["ks"], c["vs"], c["np_"], c["page"], B, H, D, c["table"], c["mp"],
                                   c["lens"], w, width, new, nmp, keep, recent, sinks, nl, kept, nw, ws, ws_bytes, None)


@pytest.mark.parametrize("kw,code", [
    (dict(w=None), NULL), (dict(new=None), NULL), (dict(nl=None), NULL), (dict(kept=None), NULL), (dict(nw=None), NULL),
    (dict(vs=None), NULL), (dict(mp=1000, width=64000, ws=None), NULL),
    (dict(keep=0), SHAPE), (dict(recent=-1), SHAPE), (dict(sinks=-1), SHAPE), (dict(recent=97), SHAPE),
    (dict(recent=101, sinks=0), SHAPE), (dict(sinks=2147483647), SHAPE), (dict(width=255), SHAPE), (dict(nmp=1), SHAPE),
    (dict(nmp=0), SHAPE), (dict(mp=1000, width=64000, ws_bytes=100), SHAPE), (dict(B=-1), SHAPE),
    (dict(page=24), UNSUP), (dict(D=100), UNSUP), (dict(w=P + 1), UNSUP), (dict(ws=P + 64), UNSUP), (dict(kp=P + 4), UNSUP),
    (dict(), DEVICE), (dict(recent=96), DEVICE), (dict(ws=None, ws_bytes=0), DEVICE),
])
def test_evict_validation(kw, code):
    assert evict_call(**kw) == code


def test_workspace_sizes():
    f = lx.kv8_attention_workspace_bytes
    assert f(2, 4096, 32, 4, 128, 64, 128) == 0              # rows enough to fill the card: not split
    assert f(1, 1, 8, 1, 128, 64, 1) == 0                    # one part's worth of keys
    for args in ((1, 1, 8, 1, 128, 64, 512), (1, 1, 64, 1, 256, 16, 512, 4000)):
        need = f(*args)
        rows = args[2]
        assert need > 0 and need % (rows * (args[4] + 2) * 4) == 0
    for bad in ((0, 1, 8, 1, 128, 64, 4), (1, 1, 7, 2, 128, 64, 4), (1, 1, 8, 1, 100, 64, 4), (1, 1, 8, 1, 128, 60, 4),
                (1, 1, 8, 1, 128, 64, 4, -1)):
        assert f(*bad) == -1
    w = lx.load().lix_kv8_token_weights_workspace_bytes
    assert w(2, 1, 16, 1, 128, 64, 8) == 0                   # one tile of rows
    assert w(64, 64, 64, 64, 128, 64, 64) == 0               # key ranges enough
    need = w(1, 2048, 32, 4, 128, 64, 64)
    assert need > 0 and need % (4 * 4096 * 4) == 0
    assert w(1, 1, 7, 2, 128, 64, 4) == -1 and w(1, 1, 8, 2, 96, 64, 4) == -1
    g = lx.load().lix_kv8_evict_workspace_bytes
    up = lambda x: (x + 255) // 256 * 256   # noqa: E731
    assert g(2, 4, 64, 512, 32768, 300, 50, 10) == 0         # rows that fit the registers of a workgroup
    assert g(2, 4, 64, 513, 40000, 300, 50, 10) == 2 * up(8 * 4) + 2 * up(8 * 240 * 4)
    assert g(2, 4, 64, 513, 40000, 60, 50, 10) == 2 * up(8 * 4)
    for bad in ((0, 4, 64, 8, 512, 5, 0, 0), (1, 1, 64, 8, 512, 5, 6, 0), (1, 1, 64, 8, 512, 5, 3, 3),
                (1, 1, 64, 8, 0, 5, 0, 0), (1, 1, 64, 8, 512, 5, -1, 0), (1, 1, 60, 8, 512, 5, 0, 0)):
        assert g(*bad) == -1


def test_bindings_refuse_tensors_before_the_library():
    cache = lx.kv8_cache(4, 2, 16, 64, device="cpu")
    assert cache.k.dtype == torch.float8_e4m3fn and cache.k_scale.shape == (4, 2)
    table, lens = torch.zeros(1, 2, dtype=torch.int32), torch.zeros(1, dtype=torch.int32)
    q = torch.zeros(1, 1, 4, 64, dtype=torch.bfloat16)
    for call in (lambda: lx.kv8_attention(q, cache, table, lens), lambda: lx.kv8_append(cache, q, q, table, lens),
                 lambda: lx.kv8_evict(cache, table, lens, torch.zeros(1, 2, 32), table, 4),
                 lambda: lx.kv8_token_weights(q, cache, table, lens, torch.zeros(1, 1, 4))):
        with pytest.raises(ValueError, match="GPU tensor"):
            call()
    with pytest.raises(ValueError, match="GPU tensor"):
        lx.rotary(q, torch.zeros(1, dtype=torch.int32), torch.zeros(8, dtype=torch.float64))
    with pytest.raises(TypeError):
        lx.rotary(q.double(), torch.zeros(1, dtype=torch.int32), torch.zeros(8, dtype=torch.float64))
    with pytest.raises(ValueError):
        lx.v4_lighting_indexer(q, q[:, :, 0], q[..., 0].float(), 1, 1, q_positions=lens)


def test_frequencies():
    f, s = lx.rotary_frequencies(64)
    assert f.dtype == torch.float64 and s == 1.0
    assert np.allclose(f.numpy(), 10000.0 ** (-np.arange(32) / 32), rtol=1e-15)
    lin, s = lx.rotary_frequencies(64, scaling="linear", factor=8.0)
    assert torch.equal(lin, f / 8) and s == 1.0
    ntk, _ = lx.rotary_frequencies(64, scaling="ntk", factor=8.0)
    # the highest frequency stays, the lowest is divided by the factor
    assert float(ntk[0]) == 1.0 and abs(float(ntk[-1] / f[-1]) - 1 / 8) < 1e-12
    for kind in ("yarn", "llama3"):
        g, s = lx.rotary_frequencies(64, scaling=kind, factor=8.0, original_max_position=4096)
        r = (g / f).numpy()
        assert r[0] == 1.0 and abs(r[-1] - 1 / 8) < 1e-12 and (np.diff(r) <= 1e-15).all()
        assert s == (0.1 * math.log(8.0) + 1.0 if kind == "yarn" else 1.0)
        turns = 4096 * f.numpy() / (2 * math.pi)
        fast, slow = (32.0, 1.0) if kind == "yarn" else (4.0, 1.0)
        assert (r[turns > 2 * fast] == 1.0).all() and np.allclose(r[turns < slow / 2], 1 / 8, rtol=1e-12)
        same, _ = lx.rotary_frequencies(64, scaling=kind, factor=1.0, original_max_position=4096)
        assert np.allclose(same.numpy(), f.numpy(), rtol=1e-15)
    for bad in (dict(rot=3), dict(rot=0), dict(rot=8, scaling="other"), dict(rot=8, scaling="yarn", factor=2.0),
                dict(rot=8, factor=0.5), dict(rot=2, scaling="ntk", factor=2.0)):
        with pytest.raises(ValueError):
            lx.rotary_frequencies(**bad)


def test_oracle_e4m3_is_torchs():
    g = np.random.default_rng(0)
    mid = (ok8.E4M3[:126] + ok8.E4M3[1:127]) / 2
    x = np.concatenate([g.normal(0, 100, 5000), ok8.E4M3[:127], mid, -mid, [0.0, -0.0, 448.0, 464.0, -1e9, np.nan]])
    x = x.astype(np.float32)
    want = torch.from_numpy(x).clamp(-448, 448).to(torch.float8_e4m3fn)
    got = ok8.e4m3_encode(x)
    assert np.array_equal(got, want.view(torch.uint8).numpy())
    assert np.array_equal(ok8.E4M3[got], want.double().numpy(), equal_nan=True)


def test_oracle_page_scale():
    for top, want in ((448.0, 1.0), (448.5, 2.0), (224.0, 0.5), (1.0, 2.0 ** -8), (0.0, 2.0 ** -60), (3e38, 2.0 ** 120)):
        assert ok8.page_scale(top) == want


def test_oracle_rotary_turns_and_returns():
    g = np.random.default_rng(1)
    x = g.normal(size=(3, 2, 2, 12))
    pos = g.integers(-50, 50, (3, 2))
    f = g.uniform(0.1, 1, 4)
    for layout in ("half", "interleaved"):
        y = orot.rotary(x, pos, f, layout, 2, 1.0)
        assert np.allclose((y ** 2).sum(-1), (x ** 2).sum(-1))             # a rotation
        assert np.allclose(orot.rotary(y, pos, f, layout, 2, 1.0, inverse=True), x)
        a = orot.rotary(orot.rotary(x, pos, f, layout, 2), pos + 1, f, layout, 2)
        assert np.allclose(a, orot.rotary(x, 2 * pos + 1, f, layout, 2))   # angles add


def test_oracle_attention_against_a_plain_softmax():
    g = np.random.default_rng(2)
    H, D, page, n = 2, 64, 16, 40
    c = {x: ok8.e4m3_encode(g.normal(0, 50, (3, H, page, D))) for x in ("k", "v")}
    c.update({x + "_scale": g.uniform(0.01, 0.02, (3, H)) for x in ("k", "v")})
    table = np.array([[2, 0, 1]])
    q = g.normal(size=(1, 5, 4, D))
    out, lse, _, _ = ok8.attention(q, c, table, [n], 0.125, [30], [4])
    for x in ("k", "v"):
        full = ok8.E4M3[c[x]] * c[x + "_scale"][..., None, None]
        c[x + "_all"] = np.concatenate([full[2], full[0], full[1]], axis=1)
    for t in range(5):
        for h in range(4):
            seen = min(n, 31 + t) if t < 4 else 0
            if not seen:
                assert (out[0, t, h] == 0).all() and lse[0, t, h] == -np.inf
                continue
            x = 0.125 * c["k_all"][h // 2, :seen] @ q[0, t, h]
            p = np.exp(x) / np.exp(x).sum()
            assert np.allclose(out[0, t, h], p @ c["v_all"][h // 2, :seen])
            assert np.allclose(lse[0, t, h], np.log(np.exp(x).sum()))
    w = ok8.token_weights(q, c, table, [n], lse, 0.125, [30], [4])
    assert np.allclose(w[0, :, :n].sum(-1), 4 * 2) and np.isnan(w[0, :, n:]).all()
