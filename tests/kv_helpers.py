"""Caches for the 8-bit cache's tests: random codes with everything a call may
not look at poisoned (NaN codes and scales in free slots and pages)."""
import numpy as np

from oracle import kv as okv


def make_cache(rng, fmt, lens, P, H, D, extra=0, spare=2, poison=True):
    """(cache, table): sequence b holds lens[b] tokens and has pages for
    `extra` more; page ids are shuffled, free columns hold -1 or ids past the
    end, free slots and pages hold NaN codes (e4m3) and NaN scales."""
    need = [(n + extra + P - 1) // P for n in lens]
    pages, width = sum(need) + spare, max(1, max(need)) + 1
    perm = rng.permutation(pages)
    table = np.where(rng.random((len(lens), width)) < 0.5, -1, pages + 5).astype(np.int32)
    c = dict(k_pages=rng.integers(0, 256, (pages, H, P, D), dtype=np.uint8),
             v_pages=rng.integers(0, 256, (pages, H, D, P), dtype=np.uint8),
             k_scales=np.exp2(rng.integers(-9, -4, (pages, H))).astype(np.float32),
             v_scales=np.exp2(rng.integers(-9, -4, (pages, H))).astype(np.float32), fmt=fmt)
    for name in ("k_pages", "v_pages"):
        x = c[name]
        if fmt == "e4m3":
            x[(x & 127) == 127] = 3
        else:
            x[x == 128] = 127
    bad = 0x7f if fmt == "e4m3" else 0x80
    used, i = set(), 0
    for b, n in enumerate(lens):
        table[b, :need[b]] = perm[i:i + need[b]]
        i += need[b]
        for col in range(need[b]):
            page, fill = table[b, col], min(max(n - col * P, 0), P)
            if poison:
                c["k_pages"][page, :, fill:] = bad
                c["v_pages"][page, :, :, fill:] = bad
            if fill:
                used.add(int(page))
    if poison:
        free = [p for p in range(pages) if p not in used]
        for name in ("k", "v"):
            c[name + "_pages"][free] = bad
            c[name + "_scales"][free] = np.nan
    return c, table


def to_device(sv, c, device="cuda"):
    import torch
    dt = torch.float8_e4m3fn if c["fmt"] == "e4m3" else torch.int8
    t = {k: torch.from_numpy(v.copy()).to(device) for k, v in c.items() if k != "fmt"}
    return sv.KVCache(t["k_pages"].view(dt), t["v_pages"].view(dt), t["k_scales"], t["v_scales"])


def to_host(cache, fmt):
    import torch
    return dict(k_pages=cache.k_pages.view(torch.uint8).cpu().numpy(),
                v_pages=cache.v_pages.view(torch.uint8).cpu().numpy(),
                k_scales=cache.k_scales.cpu().numpy(), v_scales=cache.v_scales.cpu().numpy(), fmt=fmt)


def canonical(codes, fmt):
    """Codes with one NaN (its sign is not specified)."""
    return np.where((codes & 127) == 127, 127, codes) if fmt == "e4m3" else codes


def attention_bounds(out, lse, mag, big, cnt, scale, D, dtype):
    """Allowed error of out and lse.

    u = 2^-24 is half a step of 32 bits.  A score is a sum of D exact products
    of 16- or 32-bit values with 8-bit codes, times factors rounded once each:
    off by at most ds = (D + 8) u times the sum of the products' magnitudes
    (`big`).  exp2 and log2 add a few u.  Every weight is then off by e^(2 ds)
    relative, its rounding to the products' type (half a step of bf16, 2^-8;
    u in 32 bits), the sums over cnt terms by cnt u of the sum of magnitudes
    (`mag`), and the output by half a step of its type."""
    u = 2.0 ** -24
    half = 2.0 ** -8 if dtype == "bf16" else u
    ds = (D + 8) * u * big
    tol_out = half * np.abs(out) + mag * (half + 2 * ds + (cnt + 16) * u)[..., None] * 1.01 + 1e-37
    fin = np.isfinite(lse)
    tol_lse = np.where(fin, ds + (cnt + 16) * u + 4 * u * np.abs(np.where(fin, lse, 0.0)), 0.0)
    return tol_out, tol_lse
