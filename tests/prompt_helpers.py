"""Bounds and inputs of the prompts' tests."""
import numpy as np

U = 2.0 ** -24  # half a step of 32 bits


def score_error(big, D):
    """Largest error of a score.  It is a sum of D products whose operands are
    bf16, products exact in 32 bits, or three bf16 pieces each, of whose nine
    products six are taken: by truncation a piece is below 2^-7 of what is
    left, so the others are below 2 * 2^-21 + 2^-28 < 2^-19 = 32 u.  Every
    addition rounds by at most u of the sum of magnitudes, and six products per
    channel are added; the factors round a few times."""
    return (6 * D + 48) * U * big


def attention_bounds(out, lse, mag, big, cnt, D, dtype):
    """Allowed error of out and lse: e^(2 ds) on every weight with ds a score's
    error, its rounding to the products' type (half a step of bf16, 2^-8; in 32
    bits the products' 32 u), six additions a term in sums over cnt terms, exp2
    and log2 a few u, and half a step of the output's type."""
    half = 2.0 ** -8 if dtype == "bf16" else 48 * U
    ds = score_error(big, D)
    tol_out = (2.0 ** -8 if dtype == "bf16" else U) * np.abs(out) + \
        mag * (half + 2 * ds + (6 * cnt + 16) * U)[..., None] * 1.01 + 1e-37
    fin = np.isfinite(lse)
    tol_lse = np.where(fin, ds + (cnt + 16) * U + 4 * U * np.abs(np.where(fin, lse, 0.0)), 0.0)
    return tol_out, tol_lse


def inputs(rng, T, Hq, H, D, dtype, fused=True, device="cuda"):
    """q, k, v on the device, slices of one projection's rows when fused, and
    their exact fp64 values."""
    import torch
    dt = torch.bfloat16 if dtype == "bf16" else torch.float32
    x = torch.from_numpy(rng.normal(size=(T, Hq + 2 * H, D)).astype(np.float32)).to(dt)
    host = x.double().numpy()
    parts = x.to(device).split((Hq, H, H), 1)
    if not fused:
        parts = [t.contiguous() for t in parts]
    return parts, (host[:, :Hq], host[:, Hq:Hq + H], host[:, Hq + H:])
