"""Inputs and comparison rules for the 8-bit cache and rotary tests.

Tolerances, from the arithmetic (u = 2^-24, one fp32 rounding):
* A score is a product over D summed in fp32, then scaled: off by at most
  (D + 4) u top, top = the row's largest scale * sum |q k|; the exponent, in
  units of log2, takes three more roundings of values up to |x| log2(e) + 16,
  and exp2 and log2 are good to 2^-22 of the result.  So a weight is off by
  d = (D + 4) u top + 4 u (top + 16) + 2^-21 of its value, and so is its sum.
* out: each weight is rounded once to fp16 (half a step: 2^-11 of it, or
  2^-25 in its unit, where the largest weight is at least 2^2: 2^-27 of it),
  sums of n products add n u at most, and the result is rounded to its type.
  |out - ref| <= mag (2^-11 + 2 d + n u) + 2^-27 n vmax + eps/2 |ref|.
* lse: d + 2^-21 + 4 u |ref|.
* token weights: ref (d + rows u) with |lse| rounded to fp32 (u |lse|).
"""

import numpy as np
import torch

U = 2.0 ** -24


def half_step(dtype):
    return torch.finfo(dtype).eps / 2


def rel_weight(top, D):
    return (D + 4) * U * top + 4 * U * (top + 16) + 2.0 ** -21


def out_tolerance(ref, mag, top, D, n, vmax, dtype):
    d = rel_weight(top, D)[..., None]
    return mag * (2.0 ** -11 + 2 * d + n * U) + 2.0 ** -27 * n * vmax + half_step(dtype) * np.abs(ref) + 1e-30


def lse_tolerance(ref, top, D):
    return rel_weight(top, D) + 2.0 ** -21 + 4 * U * np.abs(np.where(np.isfinite(ref), ref, 0.0))


def close(got, ref, tol, what):
    """Same values within tol; the same NaN, infinities and shapes."""
    got = np.asarray(got, dtype=np.float64)
    assert got.shape == ref.shape, what
    assert np.array_equal(np.isnan(got), np.isnan(ref)), f"{what}: NaN in other places"
    inf = np.isinf(ref)
    assert np.array_equal(got[inf], ref[inf]) and not np.isinf(got[~inf]).any(), f"{what}: infinities"
    ok = np.isfinite(ref)
    if not ok.any():
        return
    over = np.abs(got[ok] - ref[ok]) - np.broadcast_to(tol, ref.shape)[ok]
    assert (over <= 0).all(), f"{what}: {int((over > 0).sum())} of {over.size} beyond tolerance, by {over.max():.3e}"


def random_cache(num_pages, H, page, D, seed, stale_nan=True):
    """uint8 codes k, v and float32 scales; a few octaves between scales."""
    g = np.random.default_rng(seed)
    c = {}
    for x in ("k", "v"):
        vals = torch.from_numpy(g.normal(0, 60, (num_pages, H, page, D)).clip(-448, 448).astype(np.float32))
        c[x] = vals.to(torch.float8_e4m3fn).view(torch.uint8).numpy().copy()
        c[x + "_scale"] = np.exp2(g.uniform(-1, 1, (num_pages, H))).astype(np.float32) / np.float32(60)
    return c


def table_for(lens, page, num_pages, max_pages, seed):
    """Distinct random pages for each sequence's tokens, -1 behind."""
    order = np.random.default_rng(seed).permutation(num_pages).tolist()
    t = np.full((len(lens), max_pages), -1, dtype=np.int32)
    for b, n in enumerate(lens):
        for i in range(-(-n // page)):
            t[b, i] = order.pop()
    return t


def spoil_behind(cache, table, lens, page):
    """NaN codes in every slot behind a sequence's end, and NaN scales on pages that no sequence has."""
    for b, n in enumerate(lens):
        if n % page:
            for x in ("k", "v"):
                cache[x][table[b, n // page], :, n % page:] = 0x7F
    used = set(table[table >= 0].ravel().tolist())
    for p in range(cache["k"].shape[0]):
        if p not in used:
            for x in ("k", "v"):
                cache[x][p] = 0xFF
                cache[x + "_scale"][p] = np.nan


def to_device(lx, cache, dev):
    t = lambda x: torch.from_numpy(np.ascontiguousarray(x)).to(dev)   # noqa: E731
    return lx.KV8Cache(t(cache["k"]).view(torch.float8_e4m3fn), t(cache["v"]).view(torch.float8_e4m3fn),
                       t(cache["k_scale"]), t(cache["v_scale"]))


def in_f64(cache):
    return {x: (v.astype(np.float64) if x.endswith("scale") else v.copy()) for x, v in cache.items()}


def ints(values, dev):
    return torch.tensor(values, dtype=torch.int32, device=dev)
