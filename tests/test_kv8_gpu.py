"""The 8-bit cache on the GPU against the float64 oracle (oracle/kv8.py)."""

import numpy as np
import pytest
import torch

import oracle.kv8 as ok8
import sparse_attention_lightning_bf16_amd as lx
from tests import kv8_cases as kc

pytestmark = pytest.mark.gpu

DEV = "cuda:0"
BF, FP = torch.bfloat16, torch.float16


def queries(B, S, Hq, D, dtype, seed):
    return torch.randn(B, S, Hq, D, generator=torch.Generator().manual_seed(seed)).to(dtype)


def check_attention(q, cache, table, lens, q_start=None, q_lens=None, ratio=1, indices=None, scale=None, what=""):
    """Runs the call on the inputs (numpy cache and lists) and compares out and lse; returns them."""
    D = q.shape[3]
    scale = D ** -0.5 if scale is None else scale
    dev = kc.to_device(lx, cache, DEV)
    idx = None if indices is None else torch.from_numpy(indices).to(DEV)
    opt = lambda x: None if x is None else kc.ints(x, DEV)   # noqa: E731
    out, lse = lx.kv8_attention(q.to(DEV), dev, torch.from_numpy(table).to(DEV), kc.ints(lens, DEV), opt(q_start),
                                opt(q_lens), ratio, scale, idx)
    torch.cuda.synchronize()
    with np.errstate(all="ignore"):
        ref, rl, mag, top = ok8.attention(q.double().numpy(), kc.in_f64(cache), table, lens, scale, q_start, q_lens,
                                          ratio, indices)
    n = max(1, table.shape[1] * cache["k"].shape[2] if indices is None else indices.shape[2])
    vmax = 448.0 * float(np.nanmax(cache["v_scale"]))
    kc.close(out.cpu().double().numpy(), ref, kc.out_tolerance(np.nan_to_num(ref), mag, top, D, n, vmax, q.dtype),
             what + " out")
    kc.close(lse.cpu().double().numpy(), rl, kc.lse_tolerance(rl, top, D), what + " lse")
    return out, lse


@pytest.mark.parametrize("B,S,Hq,H,D,page,lens,dtype", [
    (1, 1, 1, 1, 64, 16, [1], BF),
    (2, 1, 8, 1, 128, 64, [15, 16], BF),
    (3, 1, 6, 2, 64, 16, [17, 0, 33], FP),
    (2, 1, 64, 8, 128, 64, [1000, 257], BF),
    (1, 1, 128, 1, 128, 32, [300], FP),           # more heads than a wave's rows
    (2, 1, 7, 7, 256, 128, [129, 500], BF),
    (1, 3, 40, 2, 256, 16, [77], FP),
    (2, 5, 12, 4, 128, 128, [640, 31], FP),
])
def test_attention_over_whole_sequences(B, S, Hq, H, D, page, lens, dtype):
    mp = max(1, -(-max(lens) // page)) + 1
    cache = kc.random_cache(B * mp + 3, H, page, D, 11)
    table = kc.table_for(lens, page, B * mp + 3, mp, 12)
    kc.spoil_behind(cache, table, lens, page)
    check_attention(queries(B, S, Hq, D, dtype, 13), cache, table, lens)


@pytest.mark.parametrize("B,S,Hq,H,D,page,lens,ratio,dtype", [
    (1, 40, 4, 2, 64, 16, [40], 1, BF),
    (2, 33, 6, 2, 128, 64, [100, 33], 1, BF),
    (3, 70, 8, 8, 128, 32, [70, 5, 0], 1, FP),    # more queries than tokens, and none
    (1, 90, 16, 1, 128, 64, [45], 4, BF),         # compressed positions: the first rows see nothing
    (2, 20, 3, 1, 256, 16, [64, 31], 2, FP),
])
def test_attention_causal(B, S, Hq, H, D, page, lens, ratio, dtype):
    mp = max(1, -(-max(lens) // page))
    cache = kc.random_cache(B * mp + 2, H, page, D, 21)
    table = kc.table_for(lens, page, B * mp + 2, mp, 22)
    kc.spoil_behind(cache, table, lens, page)
    q_lens = [min(S, n * ratio) for n in lens]
    q_start = [n * ratio - m for n, m in zip(lens, q_lens)]
    out, lse = check_attention(queries(B, S, Hq, D, dtype, 23), cache, table, lens, q_start, q_lens, ratio)
    for b, m in enumerate(q_lens):                # padded queries
        assert bool((out[b, m:] == 0).all()) and bool((lse[b, m:] == float("-inf")).all())


def test_attention_with_positions_outside_the_sequence():
    # queries before the first token and far behind the last one
    cache = kc.random_cache(4, 1, 16, 64, 31)
    table = kc.table_for([20, 20, 20], 16, 4 + 2, 2, 32) % 4
    check_attention(queries(3, 4, 2, 64, BF, 33), cache, table, [20, 20, 20],
                    [-3, 2147483640, -2147483648], [4, 9, -1], 1)


@pytest.mark.parametrize("B,S,Hq,H,D,page,lens,topk,dtype", [
    (1, 1, 1, 1, 64, 16, [40], 1, BF),
    (2, 3, 64, 1, 128, 64, [200, 90], 50, BF),
    (2, 5, 12, 4, 64, 16, [100, 33], 33, FP),
    (1, 9, 20, 2, 256, 32, [70], 200, BF),        # more entries than tokens
    (1, 2, 8, 1, 128, 128, [4000], 1537, FP),
])
@pytest.mark.parametrize("causal", [False, True])
def test_attention_at_given_tokens(B, S, Hq, H, D, page, lens, topk, dtype, causal):
    mp = -(-max(lens) // page)
    cache = kc.random_cache(B * mp + 2, H, page, D, 41)
    table = kc.table_for(lens, page, B * mp + 2, mp, 42)
    kc.spoil_behind(cache, table, lens, page)
    g = np.random.default_rng(43)
    idx = g.integers(-3, max(lens) + 5, (B, S, topk)).astype(np.int32)
    idx[:, -1, topk // 2:] = -1                   # padding
    idx[0, 0, :] = np.where(g.random(topk) < 0.5, idx[0, 0, 0], idx[0, 0, :])      # a token listed many times
    if S > 2:
        idx[:, 1, :] = -1                         # nothing listed
    q_start = [n - S for n in lens] if causal else None
    check_attention(queries(B, S, Hq, D, dtype, 44), cache, table, lens, q_start, None, 1, idx)


def test_attention_ignores_entries_that_are_no_page():
    lens, page = [100, 64], 16
    cache = kc.random_cache(16, 2, page, 64, 51)
    table = kc.table_for(lens, page, 16, 7, 52)
    table[0, 1], table[0, 6], table[1, 0], table[1, 2] = -1, 16, 2147483647, -2147483648
    q = queries(2, 1, 4, 64, BF, 53)
    check_attention(q, cache, table, lens)
    idx = np.arange(2 * 120, dtype=np.int32).reshape(2, 1, 120) % 120
    check_attention(q, cache, table, lens, indices=idx)
    check_attention(queries(2, 30, 4, 64, BF, 54), cache, table, lens, [70, 34], None, 1)


def test_attention_with_no_page_at_all():
    cache = kc.random_cache(2, 1, 16, 64, 55)
    table = np.full((1, 2), -1, dtype=np.int32)
    out, lse = check_attention(queries(1, 1, 3, 64, BF, 56), cache, table, [32])
    assert bool((out == 0).all()) and bool((lse == float("-inf")).all())


@pytest.mark.parametrize("D", [64, 128, 256])
def test_a_nan_reaches_only_the_queries_that_see_it(D):
    lens, page, S = [64], 16, 40
    cache = kc.random_cache(4, 1, page, D, 61)
    table = kc.table_for(lens, page, 4, 4, 62)
    cache["v"][table[0, 2], 0, 5, D // 2 + 3] = 0xFF        # token 37
    cache["k"][table[0, 3], 0, 9, 1] = 0x7F                 # token 57
    out, lse = check_attention(queries(1, S, 3, D, BF, 63), cache, table, lens, [24], None, 1)
    seen = 24 + np.arange(S) + 1
    assert np.array_equal(torch.isnan(out[0, :, 0, D // 2 + 3]).cpu().numpy(), seen > 37)
    assert np.array_equal(torch.isnan(lse[0, :, 0]).cpu().numpy(), seen > 57)


def test_attention_with_scales_of_any_size():
    lens, page = [160], 16
    cache = kc.random_cache(10, 1, page, 64, 71)
    table = kc.table_for(lens, page, 10, 10, 72)
    for i, e in enumerate([0, 30, -60, 20, -3, 100, 0, -100, 5, 101]):
        cache["v_scale"][table[0, i]] = 2.0 ** e
    cache["v_scale"][table[0, 1]] = 0.0
    cache["k_scale"][table[0, 4]] = 0.0
    check_attention(queries(1, 1, 5, 64, BF, 73), cache, table, lens)
    lens = [30]                                             # every scale zero
    cache["v_scale"][:], cache["k_scale"][:] = 0.0, 0.0
    check_attention(queries(1, 1, 5, 64, BF, 74), cache, table, lens)


def test_attention_with_scores_of_any_size():
    lens, page = [96], 32
    cache = kc.random_cache(3, 1, page, 64, 75)
    table = kc.table_for(lens, page, 3, 3, 76)
    q = queries(1, 6, 2, 64, BF, 77)
    q[0, 0] *= 0.0
    q[0, 1] *= 50.0
    q[0, 2, 0, 5] = float("nan")
    check_attention(q, cache, table, lens)
    check_attention(q, cache, table, lens, scale=0.0)


def test_attention_takes_strided_queries():
    lens, page, B, S, Hq, D = [70, 50], 16, 2, 3, 4, 64
    cache = kc.random_cache(10, 2, page, D, 81)
    table = kc.table_for(lens, page, 10, 5, 82)
    dev = kc.to_device(lx, cache, DEV)
    wide = queries(B, S, 3 * Hq, D + 8, BF, 83).to(DEV)
    q = wide[:, :, Hq:2 * Hq, 8:]
    args = (dev, torch.from_numpy(table).to(DEV), kc.ints(lens, DEV))
    got, want = lx.kv8_attention(q, *args), lx.kv8_attention(q.contiguous(), *args)
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    sbh = q.contiguous().transpose(0, 1).contiguous().transpose(0, 1)      # sequence first in memory
    got = lx.kv8_attention(sbh, *args)
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    one = q[:1, :1].expand(B, S, Hq, D)                                    # broadcast
    got, want = lx.kv8_attention(one, *args), lx.kv8_attention(one.contiguous(), *args)
    assert torch.equal(got[0], want[0])


@pytest.mark.parametrize("S", [1, 64])
def test_pages_beyond_four_gigabytes(S):
    # only the last pages of a pool of more than 2^32 bytes are used
    H, page, D = 8, 64, 128
    num = (1 << 32) // (H * page * D) + 40
    small = kc.random_cache(8, H, page, D, 91)
    k = torch.zeros(num, H, page, D, dtype=torch.uint8, device=DEV)
    v = torch.zeros(num, H, page, D, dtype=torch.uint8, device=DEV)
    ks, vs = torch.zeros(num, H, device=DEV), torch.zeros(num, H, device=DEV)
    for pool, x in ((k, "k"), (v, "v"), (ks, "k_scale"), (vs, "v_scale")):
        pool[-8:] = torch.from_numpy(small[x]).to(DEV)
    big = lx.KV8Cache(k.view(torch.float8_e4m3fn), v.view(torch.float8_e4m3fn), ks, vs)
    table = kc.table_for([400], page, 8, 7, 92)
    q = queries(1, S, 16, D, BF, 93).to(DEV)
    start = kc.ints([400 - S], DEV)
    idx = torch.arange(0, 400, 3, dtype=torch.int32, device=DEV).expand(1, S, 134).contiguous()
    dev, lens = kc.to_device(lx, small, DEV), kc.ints([400], DEV)
    at = torch.from_numpy(table).to(DEV)
    far = at + (num - 8)
    far[at < 0] = -1
    for more in ({}, {"topk_indices": idx}):
        want = lx.kv8_attention(q, dev, at, lens, start, **more)
        got = lx.kv8_attention(q, big, far, lens, start, **more)
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    lse = want[1]
    assert torch.equal(lx.kv8_token_weights(q, big, far, lens, lse, start),
                       lx.kv8_token_weights(q, dev, at, lens, lse, start))
    new = torch.randn(1, 100, H, D, device=DEV, dtype=BF)
    lx.kv8_append(big, new, new, far, kc.ints([300], DEV))
    lx.kv8_append(dev, new, new, at, kc.ints([300], DEV))
    assert torch.equal(k[-8:], dev.k.view(torch.uint8)) and torch.equal(vs[-8:], dev.v_scale)


def test_attention_is_the_same_on_every_call_and_in_any_split():
    lens, page = [3000], 64
    cache = kc.random_cache(50, 1, page, 128, 101)
    table = kc.table_for(lens, page, 50, 47, 102)
    dev = kc.to_device(lx, cache, DEV)
    args = (dev, torch.from_numpy(table).to(DEV), kc.ints(lens, DEV))
    q = queries(1, 1, 8, 128, BF, 103).to(DEV)
    need = lx.kv8_attention_workspace_bytes(1, 1, 8, 1, 128, page, 47)
    assert need > 0
    first = lx.kv8_attention(q, *args)
    ws = torch.full((need,), 255, dtype=torch.uint8, device=DEV)
    for _ in range(3):
        again = lx.kv8_attention(q, *args, workspace=ws)
        assert torch.equal(first[0], again[0]) and torch.equal(first[1], again[1])


# ------------------------------------------------------------------ append

def append_case(B, S, H, D, page, lens, new_lens, dtype, seed, spread=6):
    g = np.random.default_rng(seed)
    mp = -(-(max(lens) + S) // page)
    cache = kc.random_cache(B * mp + 2, H, page, D, seed)
    total = [n + S for n in lens]
    table = kc.table_for(total, page, B * mp + 2, mp, seed + 1)
    shape = (B, S, H, D)
    k, v = (torch.from_numpy((g.normal(0, 1, shape) * np.exp2(g.uniform(-spread, spread, (B, S, H, 1))))
                             .astype(np.float32)).to(dtype) for _ in range(2))
    return cache, table, k, v, lens, new_lens


def check_append(cache, table, k, v, lens, new_lens):
    dev = kc.to_device(lx, cache, DEV)
    lx.kv8_append(dev, k.to(DEV), v.to(DEV), torch.from_numpy(table).to(DEV), kc.ints(lens, DEV),
                  None if new_lens is None else kc.ints(new_lens, DEV))
    torch.cuda.synchronize()
    want = kc.in_f64(cache)
    with np.errstate(all="ignore"):
        ok8.append(want, k.double().numpy(), v.double().numpy(), table, lens, new_lens)
    for x in ("k", "v"):
        got, ref = getattr(dev, x).view(torch.uint8).cpu().numpy(), want[x]
        nan = (got & 0x7F == 0x7F) & (ref & 0x7F == 0x7F)
        zero = (got & 0x7F == 0) & (ref & 0x7F == 0)
        assert np.array_equal(got[~nan & ~zero], ref[~nan & ~zero]), x
        assert np.array_equal(getattr(dev, x + "_scale").cpu().numpy().astype(np.float64), want[x + "_scale"],
                              equal_nan=True), x
    return dev


@pytest.mark.parametrize("B,S,H,D,page,lens,new_lens,dtype", [
    (1, 1, 1, 64, 16, [0], None, BF),
    (3, 1, 2, 128, 64, [63, 64, 65], None, BF),
    (4, 1, 5, 64, 16, [15, 0, 100, 31], [1, 0, 1, 1], FP),
    (2, 50, 2, 128, 32, [7, 64], [50, 33], FP),
    (2, 300, 1, 256, 128, [100, 0], [300, 0], BF),
    (1, 17, 3, 256, 16, [5], [-4], BF),                     # clamped to none
    (1, 17, 3, 64, 16, [5], [99], BF),                      # clamped to S
])
def test_append_matches_oracle(B, S, H, D, page, lens, new_lens, dtype):
    check_append(*append_case(B, S, H, D, page, lens, new_lens, dtype, 201))


def test_append_keeps_special_values():
    cache, table, k, v, lens, _ = append_case(1, 40, 1, 64, 16, [3], None, BF, 211)
    k[0, 2, 0, 3], k[0, 2, 0, 4], k[0, 20, 0, 0] = float("inf"), float("-inf"), float("nan")
    v[0, 13:29] = 0.0                                       # a page of zeros: the smallest scale
    v[0, 29:] = 2.0 ** -130                                 # below the smallest scale
    k[0, 29:] = 3.0e38
    check_append(cache, table, k, v, lens, None)


def test_append_drops_tokens_without_a_page():
    cache, table, k, v, lens, _ = append_case(2, 40, 2, 64, 16, [10, 20], None, BF, 221)
    table[0, 1], table[1, 2] = -1, cache["k"].shape[0]
    check_append(cache, table, k, v, lens, None)
    check_append(cache, table, k, v, [10, 10 ** 9], None)   # behind the table's end
    check_append(cache, table, k, v, [-5, table.shape[1] * 16 - 3], None)


def test_append_twice_changes_nothing_and_takes_strides():
    cache, table, k, v, lens, new = append_case(2, 21, 3, 128, 32, [40, 9], [21, 8], FP, 231)
    once = check_append(cache, table, k, v, lens, new)
    both = torch.cat([k, v], 2).to(DEV)
    dev = kc.to_device(lx, cache, DEV)
    for _ in range(2):
        lx.kv8_append(dev, both[:, :, :3], both[:, :, 3:], torch.from_numpy(table).to(DEV), kc.ints(lens, DEV),
                      kc.ints(new, DEV))
    for a, b in zip(dev, once):
        assert torch.equal(a.view(torch.uint8), b.view(torch.uint8))


def test_append_one_by_one_holds_every_token_to_half_a_step():
    # a page's scale grows while it fills; codes move by powers of two
    B, S, H, D, page = 1, 64, 1, 64, 32
    cache, table, k, v, lens, _ = append_case(B, S, H, D, page, [0], None, BF, 241, spread=3)
    dev = kc.to_device(lx, cache, DEV)
    at = torch.from_numpy(table).to(DEV)
    for t in range(S):
        lx.kv8_append(dev, k[:, t:t + 1].to(DEV), v[:, t:t + 1].to(DEV), at, kc.ints([t], DEV))
    for x, src in (("k", k), ("v", v)):
        codes, scale = getattr(dev, x).view(torch.uint8).cpu().numpy(), getattr(dev, x + "_scale").cpu().numpy()
        for t in range(S):
            pid = table[0, t // page]
            s = float(scale[pid, 0])
            got = ok8.E4M3[codes[pid, 0, t % page]] * s
            want = src[0, t, 0].double().numpy()
            # one rounding of the value, and below e4m3's normal range of the final scale at most one
            # more for each time the scale grew, each half of its smallest step then (a geometric sum)
            assert (np.abs(got - want) <= np.maximum(2.0 ** -4 * np.abs(want), 2.0 ** -9 * s)).all(), (x, t)


# ------------------------------------------------------------------ token weights

@pytest.mark.parametrize("B,S,Hq,H,D,page,lens,ratio,dtype", [
    (1, 1, 1, 1, 64, 16, [1], 0, BF),
    (2, 1, 16, 2, 128, 64, [300, 65], 0, BF),
    (3, 1, 40, 1, 64, 32, [64, 0, 31], 0, FP),
    (2, 37, 6, 2, 128, 16, [120, 20], 1, BF),
    (1, 50, 5, 5, 256, 64, [190], 1, FP),
    (1, 60, 8, 1, 128, 32, [20], 4, BF),
])
def test_token_weights_match_oracle(B, S, Hq, H, D, page, lens, ratio, dtype):
    mp = max(1, -(-max(lens) // page)) + 1
    cache = kc.random_cache(B * mp + 2, H, page, D, 301)
    table = kc.table_for(lens, page, B * mp + 2, mp, 302)
    kc.spoil_behind(cache, table, lens, page)
    q = queries(B, S, Hq, D, dtype, 303)
    q_lens = q_start = None
    if ratio:
        q_lens = [min(S, n * ratio) for n in lens]
        q_start = [n * ratio - m for n, m in zip(lens, q_lens)]
    r = max(1, ratio)
    scale = D ** -0.5
    _, rl, _, top = ok8.attention(q.double().numpy(), kc.in_f64(cache), table, lens, scale, q_start, q_lens, r)
    lse32 = rl.astype(np.float32)
    want = ok8.token_weights(q.double().numpy(), kc.in_f64(cache), table, lens, lse32.astype(np.float64), scale,
                             q_start, q_lens, r)
    dev = kc.to_device(lx, cache, DEV)
    opt = lambda x: None if x is None else kc.ints(x, DEV)   # noqa: E731
    width = mp * page + 5
    out = torch.full((B, H, width), -7.0, device=DEV)
    args = (q.to(DEV), dev, torch.from_numpy(table).to(DEV), kc.ints(lens, DEV), torch.from_numpy(lse32).to(DEV),
            opt(q_start), opt(q_lens), r)
    lx.kv8_token_weights(*args, out=out)
    got = out.cpu().double().numpy()
    assert (got[..., mp * page:] == -7.0).all()
    got = got[..., :mp * page]
    behind = np.isnan(want)
    assert (got[behind] == -7.0).all()                       # entries behind the sequence are left as they were
    lmax = np.abs(rl[np.isfinite(rl)]).max() if np.isfinite(rl).any() else 0.0
    tol = np.nan_to_num(want) * (kc.rel_weight(top.max(), D) + 4 * kc.U * lmax + S * Hq * kc.U) + 1e-30
    kc.close(got[~behind], want[~behind], tol[~behind], "weights")
    lx.kv8_token_weights(*args, out=out, accumulate=True)
    twice = out.cpu().double().numpy()[..., :mp * page]
    assert np.array_equal(twice[~behind], 2 * got[~behind]) and (twice[behind] == -7.0).all()
    fresh = lx.kv8_token_weights(*args).cpu().double().numpy()
    assert np.array_equal(fresh[~behind], got[~behind]) and (fresh[behind] == 0).all()


def test_token_weights_of_a_query_sum_to_one():
    lens, page = [500, 123], 64
    cache = kc.random_cache(20, 2, page, 128, 311)
    table = kc.table_for(lens, page, 20, 8, 312)
    dev = kc.to_device(lx, cache, DEV)
    at, n = torch.from_numpy(table).to(DEV), kc.ints(lens, DEV)
    q = queries(2, 9, 8, 128, BF, 313).to(DEV)
    start = kc.ints([491, 114], DEV)
    _, lse = lx.kv8_attention(q, dev, at, n, start)
    w = lx.kv8_token_weights(q, dev, at, n, lse, start)
    # 9 queries x 4 heads; each sum of weights is off by the weights' error twice (lse has it too)
    assert torch.allclose(w.double().sum(-1), torch.full((2, 2), 36.0, dtype=torch.float64, device=DEV), rtol=2e-5)


# ------------------------------------------------------------------ evict

@pytest.mark.parametrize("B,H,D,page,lens,keep,recent,sinks,ties", [
    (1, 1, 64, 16, [1], 1, 0, 0, False),
    (2, 2, 128, 64, [300, 80], 100, 10, 4, False),
    (3, 1, 64, 16, [50, 51, 0], 50, 0, 0, True),
    (2, 3, 64, 16, [77, 200], 40, 36, 4, True),              # none by weight
    (2, 1, 256, 32, [130, 90], 33, 1, 0, True),
    (1, 2, 128, 128, [2500], 700, 100, 16, True),            # rows beyond 2048
    (1, 1, 64, 32, [40], 1000, 100, 4, False),               # nothing to cut
])
def test_evict_matches_oracle(B, H, D, page, lens, keep, recent, sinks, ties):
    mp, np_ = -(-max(lens) // page) + 1, -(-keep // page)
    total = B * (mp + np_)
    cache = kc.random_cache(total, H, page, D, 401)
    full = kc.table_for([mp * page + np_ * page] * B, page, total, mp + np_, 402)
    table, new_table = np.ascontiguousarray(full[:, :mp]), np.ascontiguousarray(full[:, mp:])
    g = np.random.default_rng(403)
    w = np.exp(g.normal(0, 2, (B, H, mp * page + 3))).astype(np.float32)
    if ties:
        w = np.round(w)
    cache["v"][table[0, 0], 0, 0, 5:9] = [0x7F, 0xFF, 0x7E, 0xFE]      # NaN stays, and counts for no scale
    cache["k_scale"][table[0, 0], 0] = 0.0
    dev = kc.to_device(lx, cache, DEV)
    new_lens, kept, new_w = lx.kv8_evict(dev, torch.from_numpy(table).to(DEV), kc.ints(lens, DEV),
                                         torch.from_numpy(w).to(DEV), torch.from_numpy(new_table).to(DEV), keep,
                                         recent, sinks)
    torch.cuda.synchronize()
    want = kc.in_f64(cache)
    rl, rk, rw = ok8.evict(want, table, lens, w, new_table, keep, recent, sinks)
    assert np.array_equal(new_lens.cpu().numpy(), rl)
    assert np.array_equal(kept.cpu().numpy(), rk)
    assert np.array_equal(new_w.cpu().numpy(), rw)
    for x in ("k", "v"):
        got, ref = getattr(dev, x).view(torch.uint8).cpu().numpy(), want[x]
        same = ((got & 0x7F == 0) & (ref & 0x7F == 0)) | ((got & 0x7F == 0x7F) & (ref & 0x7F == 0x7F))
        assert np.array_equal(got[~same], ref[~same]), x
        assert np.array_equal(getattr(dev, x + "_scale").cpu().numpy().astype(np.float64), want[x + "_scale"]), x


@pytest.mark.parametrize("width,keep", [(9000, 2000), (40000, 5000)])
def test_evict_of_long_rows_keeps_the_heaviest(width, keep):
    # lengths of each route of the row selection, compared with a stable sort
    H, page, D = 2, 64, 64
    mp, nk = -(-width // page), -(-keep // page)
    lens = [width, width // 2]
    cache = lx.kv8_cache(2 * (mp + nk), H, page, D, DEV)
    pages = torch.arange(2 * (mp + nk), dtype=torch.int32, device=DEV).view(2, -1)
    table, new = pages[:, :mp].contiguous(), pages[:, mp:].contiguous()
    g = torch.Generator().manual_seed(411)
    w = torch.randint(0, 50, (2, H, mp * page), generator=g).float()
    new_lens, kept, new_w = lx.kv8_evict(cache, table, kc.ints(lens, DEV), w.to(DEV), new, keep, 100, 8)
    assert new_lens.tolist() == [min(n, keep) for n in lens]
    for b, n in enumerate(lens):
        for h in range(H):
            x = w[b, h, :n].clone()
            x[:8], x[n - 100:] = 1e9, 1e9
            want = torch.sort(x, descending=True, stable=True).indices[:keep].sort().values
            assert torch.equal(kept[b, h].cpu().long(), want)
            assert torch.equal(new_w[b, h].cpu(), w[b, h][want])


def test_evict_into_entries_that_are_no_page_writes_nothing_there():
    H, page, D = 1, 16, 64
    cache = kc.random_cache(8, H, page, D, 421)
    table = np.array([[0, 1, 9, 3]], dtype=np.int32)
    new_table = np.array([[4, -1, 8]], dtype=np.int32)
    w = np.arange(64, dtype=np.float32).reshape(1, 1, 64)
    dev = kc.to_device(lx, cache, DEV)
    lx.kv8_evict(dev, torch.from_numpy(table).to(DEV), kc.ints([64], DEV), torch.from_numpy(w).to(DEV),
                 torch.from_numpy(new_table).to(DEV), 40)
    want = kc.in_f64(cache)
    ok8.evict(want, table, [64], w, new_table, 40)
    for x in ("k", "v"):
        got, ref = getattr(dev, x).view(torch.uint8).cpu().numpy(), want[x]
        zero = (got & 0x7F == 0) & (ref & 0x7F == 0)
        assert np.array_equal(got[~zero], ref[~zero])


# ------------------------------------------------------------------ together

def test_indexer_selection_attention_weights_and_eviction_together():
    """Rotated index keys select tokens; the cache is filled, read at them, weighed and cut; decoding goes on."""
    S, B, Hi, Di, Hq, H, D, page, topk, keep = 96, 2, 16, 64, 8, 2, 64, 16, 24, 40
    g = torch.Generator().manual_seed(501)
    rnd = lambda *s: torch.randn(*s, generator=g).to(BF)   # noqa: E731
    iq, ik, iw = rnd(S, B, Hi, Di), rnd(S, B, Di), torch.randn(S, B, Hi, generator=g)
    f, scale = lx.rotary_frequencies(32, scaling="yarn", factor=4.0, original_max_position=64, device=DEV)
    how = lx.Rotary(f, "interleaved", 32, scale)
    _, idx = lx.v4_lighting_indexer(iq.to(DEV), ik.to(DEV), iw.to(DEV), 1, topk, rotary=how)
    pos = torch.arange(S, dtype=torch.int32, device=DEV)
    q, k, v = rnd(B, S, Hq, D), rnd(B, S, H, D), rnd(B, S, H, D)
    qr = lx.rotary(q.to(DEV), pos[None], f, "interleaved", 0, 1.0)
    kr = lx.rotary(k.to(DEV), pos[None], f, "interleaved", 0, 1.0)

    mp, nk = S // page + 1, -(-keep // page) + 1
    cache = lx.kv8_cache(B * (mp + nk), H, page, D, DEV)
    pages = torch.randperm(B * (mp + nk), generator=g).to(torch.int32).view(B, -1).to(DEV)
    table, new_table = pages[:, :mp].contiguous(), pages[:, mp:].contiguous()
    lens = kc.ints([0, 0], DEV)
    for a in range(0, S, 37):                                # three chunks
        lx.kv8_append(cache, kr[:, a:a + 37], v.to(DEV)[:, a:a + 37], table, lens)
        lens = lens + min(37, S - a)
    start = kc.ints([0, 0], DEV)
    out, _ = lx.kv8_attention(qr, cache, table, lens, start, topk_indices=idx)
    full, lse = lx.kv8_attention(qr, cache, table, lens, start)
    w = lx.kv8_token_weights(qr, cache, table, lens, lse, start)
    new_lens, kept, _ = lx.kv8_evict(cache, table, lens, w, new_table, keep, 8, 2)
    last, _ = lx.kv8_attention(qr[:, -1:], cache, new_table, new_lens)

    # the oracle on the same cache bytes
    host = {"k": cache.k.view(torch.uint8).cpu().numpy(), "v": cache.v.view(torch.uint8).cpu().numpy(),
            "k_scale": cache.k_scale.cpu().numpy(), "v_scale": cache.v_scale.cpu().numpy()}
    c64, at = kc.in_f64(host), table.cpu().numpy()
    qd = qr.cpu().double().numpy()
    for got, more in ((out, dict(indices=idx.cpu().numpy())), (full, {})):
        ref, _, mag, top = ok8.attention(qd, c64, at, [S, S], D ** -0.5, [0, 0], None, 1, **more)
        tol = kc.out_tolerance(ref, mag, top, D, S, 448 * host["v_scale"].max(), BF)
        kc.close(got.cpu().double().numpy(), ref, tol, "together")
    ref, _, mag, top = ok8.attention(qd[:, -1:], c64, new_table.cpu().numpy(), [keep, keep], D ** -0.5)
    tol = kc.out_tolerance(ref, mag, top, D, S, 448 * host["v_scale"].max(), BF)
    kc.close(last.cpu().double().numpy(), ref, tol, "after eviction")
    # kept rows are the old ones: the values they stand for agree to one rounding of e4m3
    for b in range(B):
        for h in range(H):
            s = int(kept[b, h, 20])
            old = ok8.E4M3[host["k"][at[b, s // page], h, s % page]] * host["k_scale"][at[b, s // page], h]
            p = int(new_table[b, 20 // page])
            new = ok8.E4M3[host["k"][p, h, 20 % page]] * host["k_scale"][p, h]
            assert (np.abs(old - new) <= np.maximum(2.0 ** -4 * np.abs(old), 2.0 ** -10 * host["k_scale"][p, h])).all()


def _decode_setup(seed):
    lens, page = [700, 90], 64
    cache = kc.random_cache(30, 2, page, 128, seed)
    table = kc.table_for([760, 150], page, 30, 12, seed + 1)
    dev = kc.to_device(lx, cache, DEV)
    return dev, torch.from_numpy(table).to(DEV), kc.ints(lens, DEV), queries(2, 1, 8, 128, BF, seed + 2).to(DEV)


def _step(cache, table, lens, q, kv, weights, new_table):
    lx.kv8_append(cache, kv[:, :, :2], kv[:, :, 2:], table, lens)
    out, lse = lx.kv8_attention(q, cache, table, lens)
    lx.kv8_token_weights(q, cache, table, lens, lse, out=weights, accumulate=True)
    return (out, lse) + lx.kv8_evict(cache, table, lens, weights, new_table, 100, 10, 4)


def test_a_captured_step_replays_with_new_inputs():
    cache, table, lens, q = _decode_setup(601)
    spare = torch.tensor([[i, i + 1] for i in (0, 2)], dtype=torch.int32, device=DEV)
    used = set(table[table >= 0].tolist())
    free = [p for p in range(30) if p not in used]
    spare = torch.tensor([free[:2], free[2:4]], dtype=torch.int32, device=DEV)
    kv = torch.randn(2, 1, 4, 128, device=DEV, dtype=BF)
    w = torch.zeros(2, 2, 12 * 64, device=DEV)
    _step(cache, table, lens, q, kv, w, spare)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    w.zero_()
    with torch.cuda.graph(graph):
        got = _step(cache, table, lens, q, kv, w, spare)
    for i in range(3):
        kv.copy_(torch.randn(2, 1, 4, 128, device=DEV, dtype=BF) * (i + 1))
        q.copy_(torch.randn(2, 1, 8, 128, device=DEV, dtype=BF))
        lens.add_(1)
        w.zero_()
        twin = lx.KV8Cache(*(x.clone() for x in cache))
        w2 = w.clone()
        graph.replay()
        torch.cuda.synchronize()
        want = _step(twin, table, lens, q, kv, w2, spare)
        torch.cuda.synchronize()
        for a, b in zip(got, want):
            assert torch.equal(a, b)
        assert torch.equal(w, w2)
        for a, b in zip(cache, twin):
            assert torch.equal(a.view(torch.uint8), b.view(torch.uint8))


def test_calls_on_two_streams_at_once():
    setups = [_decode_setup(701), _decode_setup(801)]
    want = [lx.kv8_attention(q, c, t, n) for c, t, n, q in setups]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in setups]
    got = []
    for st, (c, t, n, q) in zip(streams, setups):
        with torch.cuda.stream(st):
            got.append([lx.kv8_attention(q, c, t, n) for _ in range(5)])
    torch.cuda.synchronize()
    for g, w in zip(got, want):
        for out, lse in g:
            assert torch.equal(out, w[0]) and torch.equal(lse, w[1])


def test_refusals_on_the_device():
    cache, table, lens, q = _decode_setup(901)
    with pytest.raises(lx.LixError):
        lx.kv8_attention(q, cache, table, lens, compress_ratio=0)
    with pytest.raises(lx.LixError):
        lx.kv8_attention(q, cache, table, lens, scale=float("nan"))
    with pytest.raises(lx.LixError):
        wide = torch.full((2, 64), -1, dtype=torch.int32, device=DEV)      # 4096 tokens: more than one part
        lx.kv8_attention(q, cache, wide, lens, workspace=torch.empty(16, dtype=torch.uint8, device=DEV))
    with pytest.raises(ValueError):
        lx.kv8_attention(q.clone().requires_grad_(), cache, table, lens)
    with pytest.raises(ValueError):
        lx.kv8_attention(q, cache, table.cpu(), lens)
    with pytest.raises(ValueError):
        lx.kv8_attention(q[..., ::2], cache, table, lens)
    odd = torch.zeros(2, 1, 8, 132, dtype=BF, device=DEV)[..., :128]
    with pytest.raises(lx.LixError):                         # rows not 16-byte aligned
        lx.kv8_attention(odd, cache, table, lens)
    w = torch.zeros(2, 2, 100, device=DEV)
    with pytest.raises(lx.LixError):                         # narrower than the table
        lx.kv8_token_weights(q, cache, table, lens, torch.zeros(2, 1, 8, device=DEV), out=w)
    with pytest.raises(lx.LixError):
        lx.kv8_evict(cache, table, lens, torch.zeros(2, 2, 768, device=DEV), table, 100, 90, 20)
