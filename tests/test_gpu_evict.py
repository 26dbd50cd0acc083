"""mla_cache_evict against the oracle's eviction: exact, whatever the lengths, ties and types."""

import ctypes

import numpy as np
import pytest
import torch

import oracle
from mla_latent_kv_35_b200 import binding as B
from gpu_util import dims, ensure_lib, status
from serving_util import DEV, bits, i32, page_table

gpu = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if torch.cuda.is_available():
        ensure_lib()
        B.mla_get_device_status()


def raw_pool(rng, d, n_pages, fp8):
    """A pool of random bits and its [row][byte] view."""
    row = 656 if fp8 else (d.d_latent + d.d_rope) * (2 if d.dtype == "bf16" else 4)
    by = rng.integers(0, 256, (n_pages, d.page_size, row), dtype=np.uint8)
    t = torch.from_numpy(by).to(DEV)
    return t if fp8 else t.view(d.torch_dtype), by


def run(d, lens, budget, w, pos=None, n_sink=0, n_recent=0, fp8=False, alias=False, seed=0, stride=None,
        keep_pos=True, extra_pages=0, shift=0):
    rng = np.random.default_rng(seed)
    nB, stride = len(lens), stride or max(max(lens), 1)
    table, n_pages = page_table(rng, lens, d.page_size, extra=extra_pages)
    pool, by = raw_pool(rng, d, n_pages, fp8)
    if shift:                                        # a pool at an odd multiple of its type's size
        store = torch.empty(pool.numel() + shift, dtype=pool.dtype, device=DEV)
        store[shift:] = pool.view(-1)
        pool = store[shift:].view(pool.shape)
    W = np.full((nB, stride), 123.0, np.float32)
    P = np.full((nB, stride), -5, np.int32)
    for b, L in enumerate(lens):
        W[b, :L] = w[b]
        P[b, :L] = np.arange(L) if pos is None else pos[b]
    wd, ld = torch.from_numpy(W).to(DEV), i32(lens)
    pd = None if pos is None else torch.from_numpy(P).to(DEV)
    nw = wd if alias else torch.full((nB, stride), 77.0, device=DEV)
    npos = (pd if alias and pd is not None else torch.full((nB, stride), 66, dtype=torch.int32, device=DEV)) if keep_pos else None
    nl = ld if alias else torch.full((nB,), 55, dtype=torch.int32, device=DEV)
    ws = torch.full((B.mla_cache_evict_workspace_size(d, nB, stride),), 0xAB, dtype=torch.uint8, device=DEV)
    args = (d, pool, n_pages, fp8, i32(table), table.shape[1], ld, nB, wd, pd, stride, i32(budget), n_sink,
            n_recent, nw, npos, nl, ws)
    B.mla_cache_evict(*args)
    assert status() == 0
    exp = by.copy()
    ew = W.copy() if alias else np.full_like(W, 77.0)
    ep = P.copy() if alias and pos is not None else np.full_like(P, 66)
    el = []
    for b, L in enumerate(lens):
        pairs, new = oracle.evict(W[b, :L], P[b, :L].tolist(), budget[b], n_sink, n_recent)
        ew[b, :new], ep[b, :new] = W[b, :new], P[b, :new]
        for to, frm in pairs:
            exp[table[b, to // d.page_size], to % d.page_size] = by[table[b, frm // d.page_size], frm % d.page_size]
            ew[b, to], ep[b, to] = W[b, frm], P[b, frm]
        el.append(new)
    np.testing.assert_array_equal(nl.cpu().numpy(), el)
    np.testing.assert_array_equal(bits(nw), ew.view(np.int32))
    if keep_pos:
        np.testing.assert_array_equal(npos.cpu().numpy(), ep)
    np.testing.assert_array_equal(pool.contiguous().view(torch.uint8).cpu().numpy().reshape(by.shape), exp)
    return el


def draw_w(rng, lens, kind):
    out = []
    for L in lens:
        if kind == "ties":
            x = rng.integers(0, 4, L).astype(np.float32)
        elif kind == "equal":
            x = np.full(L, 0.25, np.float32)
        elif kind == "odd":
            x = rng.choice(np.array([0.0, -0.0, np.inf, -np.inf, np.nan, -np.nan, 1e-45, -1e-45, 1.0, -1.0,
                                     3.4e38, -3.4e38], np.float32), L)
        else:
            x = np.exp(2.5 * rng.standard_normal(L)).astype(np.float32)
        out.append(x)
    return out


LENS = [0, 1, 2, 31, 32, 33, 63, 64, 65, 700, 1023, 1025]


@gpu
@pytest.mark.parametrize("kind", ["spread", "ties", "equal", "odd"])
@pytest.mark.parametrize("placed", [False, True])
def test_small_lengths(kind, placed):
    rng = np.random.default_rng(1)
    w = draw_w(rng, LENS, kind)
    pos = [rng.permutation(3 * L)[:L] for L in LENS] if placed else None
    d = dims("bf16")
    for frac in (0.0, 0.5, 0.97, 2.0):
        run(d, LENS, [int(L * frac) for L in LENS], w, pos, 2, 5)
    run(d, LENS, [L - 1 for L in LENS], w, pos, 0, 0)             # -1 counts as 0
    run(d, LENS, [-3] * len(LENS), w, pos, 0, 0)
    run(d, LENS, [0] * len(LENS), w, pos, 10 ** 6, 0)             # nothing is free
    run(d, LENS, [0] * len(LENS), w, pos, 0, 2 ** 31 - 1)


@gpu
@pytest.mark.parametrize("stride,kind", [(70, "spread"), (70, "ties"), (70, "equal"), (70, "odd"), (4097, "spread"),
                                         (9000, "ties"), (40000, "odd")])
@pytest.mark.parametrize("alias", [False, True])
def test_a_few_leave(kind, stride, alias):
    """The numbers around which sequences turn from one selection to the other, in one batch; with
    fewer free slots than should leave, the slots behind the new end leaving, and none free."""
    rng = np.random.default_rng(13)
    lens = [stride, stride - 1, 5, 4, 1, 3, 0]
    w = draw_w(rng, lens, kind)
    pos = [rng.permutation(3 * L)[:L] for L in lens]
    d = dims("bf16", dc=8, dr=0, page=16)
    run(d, lens, [L - 1 for L in lens], w, pos, 0, 0, alias=alias)
    run(d, lens, [L - 3 for L in lens], w, pos, 4, 3, alias=alias)
    run(d, lens, [L - 1 - b % 5 for b, L in enumerate(lens)], w, None, 0, 1, alias=alias)
    for b, L in enumerate(lens):                       # the lightest ones last
        w[b][max(0, L - 3):] = -np.inf
    for drop in (2, 3, 4):
        run(d, lens, [L - drop for L in lens], w, None, 0, 0, alias=alias)
    run(d, lens, [L - 3 for L in lens], w, None, 0, 2, alias=alias)
    run(d, lens, [L - 3 for L in lens], w, None, stride - 2, 0, alias=alias)          # two free
    run(d, lens, [L - 3 for L in lens], w, None, stride, 0, alias=alias)              # none


@gpu
@pytest.mark.parametrize("n_recent", [0, 1, 7, 2 ** 31 - 1])
def test_the_last_position_there_is(n_recent):
    rng = np.random.default_rng(12)
    lens = [40, 9000]
    pos = [2 ** 31 - 1 - rng.permutation(2 * L)[:L] for L in lens]
    pos[0][5] = 2 ** 31 - 1
    run(dims("bf16"), lens, [10, 4000], draw_w(rng, lens, "spread"), pos, 3, n_recent)


@gpu
@pytest.mark.parametrize("stride", [4096, 4097, 9000, 20000, 70000])
@pytest.mark.parametrize("kind", ["spread", "ties", "odd"])
def test_clusters(stride, kind):
    """1 to 8 blocks per sequence; lengths from none to the whole stride."""
    rng = np.random.default_rng(stride)
    d = dims("bf16", dc=8, dr=0, page=16)
    lens = [stride, stride - 1, 5, 0, stride // 3]
    w = draw_w(rng, lens, kind)
    run(d, lens, [L // 2 for L in lens], w, None, 3, 40, stride=stride)
    pos = [rng.permutation(2 * L)[:L] for L in lens]
    run(d, lens, [L - min(L, 7) for L in lens], w, pos, 3, 40, stride=stride, alias=True)


@gpu
@pytest.mark.parametrize("dtype,fp8,kw", [("bf16", False, {}), ("f32", False, {}), ("bf16", True, {}),
                                          ("f32", False, dict(dc=5, dr=2, page=3)),
                                          ("bf16", False, dict(dc=7, dr=2, page=16))])
@pytest.mark.parametrize("alias", [False, True])
def test_types_widths_and_aliases(dtype, fp8, kw, alias):
    rng = np.random.default_rng(3)
    d = dims(dtype, **kw)
    lens = [300, 1, 129]
    w = draw_w(rng, lens, "ties")
    pos = [rng.permutation(L) for L in lens]
    run(d, lens, [100, 1, 128], w, pos, 1, 3, fp8=fp8, alias=alias, stride=333, extra_pages=2)
    run(d, lens, [100, 0, 64], w, None, 1, 3, fp8=fp8, alias=alias, keep_pos=False)


@gpu
def test_pool_off_a_16_byte_boundary():
    rng = np.random.default_rng(4)
    w = draw_w(rng, [200, 90], "spread")
    run(dims("bf16"), [200, 90], [77, 45], w, shift=1)


@gpu
def test_one_long_sequence():
    rng = np.random.default_rng(5)
    L = 300001                                       # larger than any block's registers or caches
    d = dims("f32", dc=4, dr=0, page=64)
    run(d, [L], [123457], draw_w(rng, [L], "spread"), None, 4, 64)


@gpu
def test_bad_lengths_and_pages_are_reported():
    d = dims("bf16", dc=8, dr=0, page=16)
    for L in (-1, 33, 49):                           # stride 48, two pages of 16
        lens = i32([20, L])
        w = torch.ones((2, 48), device=DEV)
        pool = torch.zeros((5, 16, 8), dtype=torch.bfloat16, device=DEV)
        nl = torch.zeros(2, dtype=torch.int32, device=DEV)
        nw = torch.zeros((2, 48), device=DEV)
        ws = torch.empty(B.mla_cache_evict_workspace_size(d, 2, 48), dtype=torch.uint8, device=DEV)
        B.mla_cache_evict(d, pool, 5, False, i32([[0, 1], [2, 3]]), 2, lens, 2, w, None, 48, i32([10, 10]), 0,
                          0, nw, None, nl, ws)
        assert status() == 5
        assert nl.tolist() == [10, L] and (nw[1] == 0).all()
    # a page outside the pool: its rows stay, the rest moves
    pool = torch.arange(5 * 16, device=DEV).bfloat16().view(5, 16, 1).repeat(1, 1, 8).contiguous()
    before = pool.clone()
    w = torch.arange(48, device=DEV).float().repeat(2, 1)
    B.mla_cache_evict(d, pool, 5, False, i32([[0, 9], [2, 3]]), 2, i32([20, 20]), 2, w, None, 48,
                      i32([10, 10]), 0, 0, nw, None, nl, ws)
    assert status() == 5
    assert torch.equal(pool[0, :6], before[0, 10:16]) is True     # moved within the good page
    assert torch.equal(pool[0, 6:], before[0, 6:])
    assert torch.equal(pool[2, :6], before[2, 10:16]) and torch.equal(pool[2, 6:10], before[3, :4])


@gpu
def test_graph_replay_evicts_in_place_step_by_step():
    rng = np.random.default_rng(6)
    d = dims("bf16", dc=8, dr=0, page=16)
    L, cut = 100, 30
    table, n_pages = page_table(rng, [L], 16)
    pool, by = raw_pool(rng, d, n_pages, False)
    W = rng.permutation(L).astype(np.float32)[None]
    wd, pd, ld, bd = torch.from_numpy(W).to(DEV), i32(np.arange(L)[None]), i32([L]), i32([L - cut])
    ws = torch.empty(B.mla_cache_evict_workspace_size(d, 1, L), dtype=torch.uint8, device=DEV)
    g = torch.cuda.CUDAGraph()
    td = i32(table)
    with torch.cuda.graph(g):
        B.mla_cache_evict(d, pool, n_pages, False, td, table.shape[1], ld, 1, wd, pd, L, bd, 0, 0, wd,
                          pd, ld, ws)
    for step in range(3):
        bd.fill_(L - cut * (step + 1))
        g.replay()
    assert status() == 0 and ld.item() == 10
    left = sorted(wd[0, :10].tolist())
    assert left == list(range(90, 100))
    rows = pool.view(torch.uint8).cpu().numpy().reshape(by.shape)
    for s in range(10):
        p = int(pd[0, s])
        assert W[0, p] == wd[0, s].item()
        np.testing.assert_array_equal(rows[table[0, s // 16], s % 16], by[table[0, p // 16], p % 16])


def test_refused_on_the_host():
    from mla_latent_kv_35_b200 import build
    build.build()
    lib = B.lib()
    x = 1 << 12

    def call(d=dims("bf16"), pool=x, n_pages=4, fp8=0, pt=x, mp=2, sl=x, nB=2, w=x, stride=100, bud=x, ns=0,
             nr=0, nw=x, nl=x, ws=x, wb=1 << 20):
        return lib.mla_cache_evict(ctypes.byref(d.c()), pool, n_pages, fp8, pt, mp, sl, nB, w, 0, stride, bud,
                                   ns, nr, nw, 0, nl, ws, wb, 0)
    assert call(nB=0, pool=0, ws=0) == 0
    for kw in (dict(pool=0), dict(pt=0), dict(sl=0), dict(w=0), dict(bud=0), dict(nw=0), dict(nl=0),
               dict(ws=0), dict(ws=x + 16), dict(wb=100), dict(nB=-1), dict(nB=65536), dict(stride=0),
               dict(n_pages=0), dict(mp=0), dict(stride=(1 << 30) + 1), dict(ns=-1), dict(nr=-1), dict(mp=1 << 30)):
        assert call(**kw) == 1, kw
    assert call(fp8=1, d=dims("f32")) == 2
    assert call(fp8=1, d=dims("bf16", dc=256)) == 2
    assert B.mla_cache_evict_workspace_size(dims("bf16"), 3, 1000) >= 3 * 1000 * 8 + 12
    assert B.mla_cache_evict_workspace_size(dims("bf16"), 3, 0) == 0


@gpu
def test_binding_refuses_wrong_tensors():
    d = dims("bf16", dc=8, dr=0, page=16)
    good = dict(pool=torch.zeros((5, 16, 8), dtype=torch.bfloat16, device=DEV), pt=i32([[0, 1], [2, 3]]),
                sl=i32([20, 20]), w=torch.ones((2, 48), device=DEV), pos=None, bud=i32([10, 10]),
                nw=torch.ones((2, 48), device=DEV), np=None, nl=i32([0, 0]),
                ws=torch.empty(B.mla_cache_evict_workspace_size(d, 2, 48), dtype=torch.uint8, device=DEV))

    def call(fp8=False, **kw):
        a = {**good, **kw}
        B.mla_cache_evict(d, a["pool"], 5, fp8, a["pt"], 2, a["sl"], 2, a["w"], a["pos"], 48, a["bud"], 0, 0,
                          a["nw"], a["np"], a["nl"], a["ws"])
    call()
    bad = [dict(pool=good["pool"][:4]), dict(pool=good["pool"].float()), dict(pt=good["pt"][:1]),
           dict(sl=good["sl"].long()), dict(w=good["w"].double()), dict(w=good["w"][:, :40].contiguous()),
           dict(pos=good["w"]), dict(bud=good["bud"].cpu()), dict(nw=good["nw"].t()), dict(nl=good["nl"][:1]),
           dict(ws=good["ws"].view(torch.int32)), dict(fp8=True)]
    for kw in bad:
        with pytest.raises(ValueError):
            call(**kw)
    with pytest.raises(B.MLAError):
        call(ws=good["ws"][256:])
    assert status() == 0
