"""Paged caches for the tests of the operators around the latent cache."""

import numpy as np
import torch

DEV = "cuda"
U = {torch.bfloat16: 2.0 ** -8, torch.float32: 2.0 ** -24}   # half a step, relative


def page_table(rng, lens, page, spare=1, extra=0):
    """Pages in random order: (table [B, max_pages + extra] int32 with -1 unused, n_pages)."""
    npg = [-(-L // page) for L in lens]
    n_pages = sum(npg) + spare
    perm = rng.permutation(n_pages).astype(np.int32)
    table = np.full((len(lens), max(max(npg), 1) + extra), -1, np.int32)
    o = 0
    for b, n in enumerate(npg):
        table[b, :n] = perm[o:o + n]
        o += n
    return table, n_pages


def paged(rng, lens, D, dtype, page=64, unused=float("nan"), **kw):
    """(pool on the device, table on the device, n_pages, rows per sequence as float64)."""
    table, n_pages = page_table(rng, lens, page, **kw)
    pool = torch.full((n_pages, page, D), unused, dtype=torch.float32)
    rows = []
    for b, L in enumerate(lens):
        r = torch.from_numpy(rng.standard_normal((L, D)).astype(np.float32)).to(dtype).float()
        for p in range(-(-L // page)):
            part = r[p * page:(p + 1) * page]
            pool[table[b, p], :len(part)] = part
        rows.append(r.double().numpy())
    return pool.to(dtype).to(DEV), torch.from_numpy(table).to(DEV), n_pages, rows


def i32(x):
    return torch.tensor(np.asarray(x), dtype=torch.int32, device=DEV)


def bits(t):
    """The tensor's raw bits as integers (NaN compares)."""
    t = t.detach().cpu().contiguous()
    return t.view({1: torch.uint8, 2: torch.int16, 4: torch.int32}[t.element_size()]).numpy()
