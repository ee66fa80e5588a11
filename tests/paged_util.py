"""Seeded paged caches, and the error bounds of single-token attention."""
import numpy as np
import torch

from oracle import fp8, paged

DTYPES = {"bf16": torch.bfloat16, "fp32": torch.float32, "e4m3": torch.uint8}


def cache_scale(amax):
    """448 * (1 / amax) in fp32, both steps rounded."""
    return np.float32(448.0) * (np.float32(1.0) / np.float32(amax))


def values(x, amax=None):
    """fp64 values a stored tensor stands for (8-bit codes with cache_scale(amax))."""
    if x.dtype == torch.uint8:
        s = np.float64(cache_scale(amax)) if amax else 1.0
        return x.cpu().view(torch.float8_e4m3fn).float().numpy().astype(np.float64) / s
    return x.detach().float().cpu().numpy().astype(np.float64)


def codes_of(x, amax):
    """e4m3 codes (uint8 array) of rows x, by the oracle's encoder."""
    return fp8.encode(x.float().numpy() * cache_scale(amax))


def stored(x, kind, amax=None):
    """A CPU tensor of fp32 numbers as the cache stores it."""
    if kind != "e4m3":
        return x.to(DTYPES[kind])
    return torch.from_numpy(codes_of(x.to(torch.bfloat16), amax))


def rows_dtype(kind):
    return torch.float32 if kind == "fp32" else torch.bfloat16


def make_table(lens, P, width, num_pages, g):
    order = torch.randperm(num_pages, generator=g)
    table = torch.full((len(lens), width), -1, dtype=torch.int32)
    at = 0
    for r, n in enumerate(lens):
        k = paged.pages_of(n, P)
        table[r, :k] = order[at:at + k].int()
        at += k
    return table, order[at:]


def make_cache(lens, Hq, Hkv, D, P, kind, seed, scale=1.0, poison=True, spare=3, width=None):
    """CPU dict of a filled cache; positions behind each length, free pages and table
    entries behind the last page hold NaN / invalid numbers when `poison`."""
    g = torch.Generator().manual_seed(seed)
    R = len(lens)
    held = [paged.pages_of(n, P) for n in lens]
    width = max(1, max(held)) + 1 if width is None else width
    num_pages = sum(held) + spare
    table, free = make_table(lens, P, width, num_pages, g)
    amax = (5.0, 4.5)
    k = torch.randn(num_pages, Hkv, P, D, generator=g) * scale
    v = torch.randn(num_pages, Hkv, P, D, generator=g) * scale
    q = (torch.randn(R, Hq, D, generator=g) * scale).to(rows_dtype(kind))
    live = torch.zeros(num_pages, P, dtype=torch.bool)
    for r, n in enumerate(lens):
        for j in range(held[r]):
            live[table[r, j].long(), :min(P, n - j * P)] = True
    ks, vs = stored(k, kind, amax[0]), stored(v, kind, amax[1])
    if poison:
        dead = ~live[:, None, :, None].expand(num_pages, Hkv, P, D)
        for x in (ks, vs):
            x[dead] = 0x7F if kind == "e4m3" else float("nan")
        for r in range(R):
            table[r, held[r]:] = 0x7FFFFFF0
    return dict(k=ks, v=vs, q=q, table=table, lens=torch.tensor(lens, dtype=torch.int32), free=free,
                amax=torch.tensor(amax) if kind == "e4m3" else None, P=P, kind=kind)


def on_gpu(c):
    return {n: x.cuda() if isinstance(x, torch.Tensor) else x for n, x in c.items()}


def reference(c, scale, pages=None):
    a = (None, None) if c["amax"] is None else c["amax"].tolist()
    return paged.decode(values(c["q"]), values(c["k"], a[0]), values(c["v"], a[1]), c["table"].numpy(),
                        c["lens"].tolist(), scale, pages)


def assert_decode(o, lse, ref, D, scale, n_max, kind, what=""):
    """Bounds of the method, per element (units of 2^-24 unless said).

    Scores: an fp32 sum of D products is off by at most (D + 2) 2^-24 sum |q k|, the
    multiplication by scale * log2 e adds 2^-22 |x|: dx.  A weight is off by dx, 2^-21
    for 2^x, and 2^-17 where the tensor cores take it as the sum of two 16-bit numbers
    (2^-9 each).  Sums over n keys run in chains of at most n / 16 + 64 additions.  The
    quotient of the weighted sum and the sum of weights has twice that, times
    sum p |v|, and is rounded once: half a step, 2^-8 for bf16 and 2^-24 for fp32."""
    ro, rl, mass, reach = ref
    dx = (D + 2) * 2.0 ** -24 * scale * reach + 2.0 ** -22 * scale * reach
    chain = (n_max / 16 + 64) * 2.0 ** -24
    weight = dx + 2.0 ** -21 + chain + (0 if kind == "fp32" else 2.0 ** -17)
    half = 2.0 ** -8 if o.dtype == torch.bfloat16 else 2.0 ** -24
    got = values(o)
    tol = half * np.abs(ro) + (1 + half) * weight[..., None] * 2 * mass
    assert np.all(np.isfinite(got)), f"{what}: not finite"
    bad = np.abs(got - ro) - tol
    assert bad.max(initial=-1.0) <= 0, f"{what}: o off by {np.abs(got - ro).max():.3e}, {bad.max():.3e} over the bound"
    gl = values(lse)
    assert np.array_equal(np.isneginf(gl), np.isneginf(rl)), f"{what}: rows without a key differ"
    seen = np.isfinite(rl)
    off = np.abs(gl[seen] - rl[seen])
    tol_l = (dx + 2.0 ** -21 + chain)[seen] + 2.0 ** -22 * np.abs(rl[seen])
    assert np.all(off <= tol_l), f"{what}: lse off by {off.max(initial=0.0):.3e}"
