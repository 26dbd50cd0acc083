"""Calls at the edges of what the operators around the cache allow: NaN among the inputs, offsets and
pages that break their rules, evictions one after the other, appends behind an eviction, outputs at odd
addresses."""

import numpy as np
import pytest
import torch

import oracle
from mla_latent_kv_35_b200 import binding as B
from mla_latent_kv_35_b200.engine import DecodePipeline, PrefillPipeline
from gpu_util import check, dims, ensure_lib, q, status, to_dev, to_np
from serving_util import DEV, bits, i32, paged
import test_gpu_attn_weights as tw
import test_gpu_chunk as tc
from test_gpu_serving import Reference, make, tokens

gpu = pytest.mark.gpu
NAN = float("nan")


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if torch.cuda.is_available():
        ensure_lib()
        B.mla_get_device_status()


@gpu
@pytest.mark.parametrize("dm,shift,T", [(256, 1, 5), (256, 2, 130), (130, 0, 3), (131, 0, 1), (133, 3, 64),
                                        (5120, 1, 2)])
def test_out_proj_at_any_address_and_width(dm, shift, T):
    """Outputs at any float's address and a model width that is no multiple of four, with and without
    a split of the product, are those of the aligned call."""
    d = dims("bf16", H=16, dm=dm)
    g = torch.Generator(device=DEV)
    g.manual_seed(dm + T)
    mk = lambda *n: torch.randn(n, generator=g, device=DEV).bfloat16()  # noqa: E731
    o, w_uv, w_o = mk(T, 16, 512), mk(16, 128, 512), mk(dm, 16 * 128)
    wide = dims("bf16", H=16, dm=-(-dm // 8) * 8)
    w_wide = torch.zeros((wide.d_model, 16 * 128), dtype=torch.bfloat16, device=DEV)
    w_wide[:dm] = w_o
    ref = torch.empty((T, wide.d_model), device=DEV)
    s = torch.empty(B.mla_out_proj_bf16_scratch_size(wide, T), dtype=torch.uint8, device=DEV)
    B.mla_out_proj_bf16(wide, o, w_uv, w_wide, s, ref, T)
    store = torch.full((T * dm + shift + 1,), 7.0, device=DEV)
    out = store[shift:shift + T * dm].view(T, dm)
    s = torch.empty(B.mla_out_proj_bf16_scratch_size(d, T), dtype=torch.uint8, device=DEV)
    B.mla_out_proj_bf16(d, o, w_uv, w_o, s, out, T)
    assert status() == 0
    assert torch.equal(out, ref[:, :dm])
    assert (store[:shift] == 7).all() and store[-1] == 7
    # and of fp32 rows, at an odd address too
    of = torch.full((T * 16 * 512 + shift,), 0.0, device=DEV)[shift:].view(T, 16, 512)
    of.copy_(o)
    out.fill_(0)
    s = torch.empty(B.mla_out_proj_scratch_size(d, T), dtype=torch.uint8, device=DEV)
    B.mla_out_proj(d, of, w_uv, w_o, s, out, T)
    assert status() == 0
    assert torch.equal(out, ref[:, :dm]) and (store[:shift] == 7).all() and store[-1] == 7


@gpu
@pytest.mark.parametrize("S_q,lens", [(1, [1, 300]), (2, [257, 513, 40])])
def test_decode_with_a_negative_scale(S_q, lens):
    """The decode takes scales below zero too; a row that sees nothing of a 256-token block keeps its
    sums.  Tolerance as in test_gpu_chunk, for fp32 arithmetic: a score of 18 products in a row and 5
    sums is off by d = 24 * 2^-24 * |scale| * sum |q k|, its exponential by 2^-17 more, and every token
    rounds o twice."""
    d = B.MLADims(16, 128, 512, 64, 128, 5120, 64, -0.3, 10000.0, "bf16")
    nB = len(lens)
    pool, table, n_pages, rows = paged(np.random.default_rng(4), lens, 576, torch.bfloat16)
    g = torch.Generator(device=DEV)
    g.manual_seed(S_q)
    qb = (0.5 * torch.randn((nB, S_q, 16, 576), generator=g, device=DEV)).bfloat16()
    o, lse = torch.empty((nB, S_q, 16, 512), device=DEV), torch.empty((nB, S_q, 16), device=DEV)
    ws = torch.empty(B.mla_decode_workspace_size(d, nB, S_q), dtype=torch.uint8, device=DEV)
    B.mla_decode(d, qb, pool, n_pages, table, table.shape[1], i32(lens), nB, S_q, 0, ws, o, lse)
    assert status() == 0
    for b, L in enumerate(lens):
        for j in range(S_q):
            k = torch.from_numpy(rows[b][:L - S_q + j + 1]).to(DEV)
            x = qb[b, j].double()
            s = x @ k.T * d.scale
            p = torch.softmax(s, 1)
            ref, A = p @ k[:, :512], p @ k[:, :512].abs()
            e = 24 * 2.0 ** -24 * abs(d.scale) * (x.abs() @ k.abs().T).amax(1)
            tol = (2 * (e + 2.0 ** -17)[:, None] + L * 2.0 ** -23) * A
            assert ((o[b, j].double() - ref).abs() <= tol).all()
            assert ((lse[b, j].double() - torch.logsumexp(s, 1)).abs() <=
                    e + 2.0 ** -16 + 2.0 ** -22 * torch.logsumexp(s, 1).abs() + L * 2.0 ** -23).all()


@gpu
@pytest.mark.parametrize("H,qs,lens", [(16, [3, 2], [200, 90]), (128, [2, 1], [300, 513]),
                                       (128, [5, 3], [300, 70])])
def test_a_nan_lse_reaches_every_token_its_query_sees(H, qs, lens):
    """One (query, head) with lse = NaN, in each form of the kernel: the tokens it sees weigh NaN, the
    later ones and the other sequence's as if that row gave nothing."""
    d = dims("bf16", H=H)
    pool, table, n_pages, rows = paged(np.random.default_rng(1), lens, 576, torch.bfloat16)
    total, cu = sum(qs), i32(np.concatenate([[0], np.cumsum(qs)]))
    qb = torch.randn((total, H, 576), device=DEV).bfloat16()
    lse = torch.full((total, H), 8.0, device=DEV)
    got = []
    for bad in (-float("inf"), NAN):
        lse[1, H - 1] = bad                            # the second query of the first sequence
        w = torch.full((2, max(lens)), 9.0, device=DEV)
        tw.call(d, qb, lse, cu, total, max(qs), pool, n_pages, table, i32(lens), None, 1.0, w)
        assert status() == 0
        got.append(w)
    see = lens[0] - qs[0] + 2
    assert got[1][0, :see].isnan().all()
    assert torch.equal(got[1][0, see:], got[0][0, see:]) and torch.equal(got[1][1], got[0][1])
    ref, tol = tw.reference(qb[:qs[0]], torch.where(lse[:qs[0]].isnan(), -float("inf"), lse[:qs[0]]), rows[0],
                            qs[0], d.scale)
    assert ((got[0][0, :lens[0]].double() - ref).abs() <= tol + 2.0 ** -23 * ref).all()


@gpu
@pytest.mark.parametrize("H,qs,lens", [(16, [3, 1], [200, 90]), (16, [1, 2], [30000, 70]),
                                       (128, [2, 3], [9000, 300]), (128, [40, 1], [5000, 20000])])
def test_a_nan_query_gives_nan_however_it_is_split(H, qs, lens):
    """Row blocks that one worker serves and ones that many share: o and lse of a query with a NaN are
    NaN, every other row keeps its bits."""
    d = dims("bf16", H=H)
    pool, table, n_pages, _ = paged(np.random.default_rng(2), lens, 576, torch.bfloat16)
    total, cu = sum(qs), i32(np.concatenate([[0], np.cumsum(qs)]))
    qb = torch.randn((total, H, 576), device=DEV).bfloat16()
    o, lse = tc.call(d, qb, cu, total, max(qs), pool, n_pages, table, i32(lens))
    qn = qb.clone()
    bad = torch.zeros((total, H), dtype=torch.bool, device=DEV)
    for u, h in ((0, 0), (total - 1, H - 1), (qs[0] - 1, H // 2)):
        qn[u, h, 7 + h] = NAN
        bad[u, h] = True
    o2, lse2 = tc.call(d, qn, cu, total, max(qs), pool, n_pages, table, i32(lens))
    assert status() == 0
    assert o2[bad].isnan().all() and lse2[bad].isnan().all()
    assert torch.equal(o2[~bad], o[~bad]) and torch.equal(lse2[~bad], lse[~bad])


@gpu
def test_chunks_that_do_not_begin_at_the_first_token():
    """cu_q ascends from 0: a cu_q that begins later breaks its rules, and nothing is written."""
    lens = [200, 300, 90]
    d = dims("bf16", H=16)
    pool, table, n_pages, _ = paged(np.random.default_rng(3), lens, 576, torch.bfloat16)
    qb = torch.randn((9, 16, 576), device=DEV).bfloat16()
    o, lse = tc.call(d, qb, i32([1, 2, 4, 5]), 9, 4, pool, n_pages, table, i32(lens))
    assert status() == 5
    assert (o == 5).all() and (lse == 5).all()
    w = torch.full((3, 300), 9.0, device=DEV)
    tw.call(d, qb, torch.full((9, 16), 8.0, device=DEV), i32([1, 2, 4, 5]), 9, 4, pool, n_pages, table, i32(lens),
            None, 1.0, w)
    assert status() == 5
    assert (w == 9).all()


@gpu
@pytest.mark.parametrize("alias", [False, True])
@pytest.mark.parametrize("bad_page", [0, 1])
@pytest.mark.parametrize("drop", [10, 3])
def test_eviction_around_a_bad_page_keeps_rows_and_books_together(alias, bad_page, drop):
    """A pair whose source or destination lies on a page outside the pool is not moved at all: the
    vacated slot keeps its row, its weight and its position."""
    d = dims("bf16", dc=8, dr=0, page=16)
    pool = torch.arange(5 * 16, device=DEV).bfloat16().view(5, 16, 1).repeat(1, 1, 8).contiguous()
    before = pool.clone()
    table = [[0, 1], [2, 3]]
    table[0][bad_page] = 9 if bad_page else -1
    W = torch.arange(48, device=DEV).float().repeat(2, 1)
    P = (torch.arange(48, device=DEV, dtype=torch.int32) * 2).repeat(2, 1)
    w, p, lens = W.clone(), P.clone(), i32([20, 20])
    nw = w if alias else torch.full((2, 48), 77.0, device=DEV)
    np_ = p if alias else torch.full((2, 48), 66, dtype=torch.int32, device=DEV)
    nl = lens if alias else i32([0, 0])
    ws = torch.empty(B.mla_cache_evict_workspace_size(d, 2, 48), dtype=torch.uint8, device=DEV)
    B.mla_cache_evict(d, pool, 5, False, i32(table), 2, lens, 2, w, p, 48, i32([20 - drop] * 2), 0, 0, nw, np_, nl,
                      ws)
    assert status() == 5
    new = 20 - drop
    assert nl.tolist() == [new, new]
    for b in range(2):
        src = list(range(new))                         # the lightest, slots 0 .. drop - 1, leave
        for k in range(drop):
            if b == 1 or (table[0][0] == 0 and (new + k < 16 or table[0][1] == 1)):
                src[k] = new + k
        assert nw[b, :new].tolist() == W[b, src].tolist()
        assert np_[b, :new].tolist() == P[b, src].tolist()
        for t in range(new):
            if table[b][t // 16] in range(5):
                assert torch.equal(pool[table[b][t // 16], t % 16], before[table[b][src[t] // 16], src[t] % 16])


@gpu
@pytest.mark.parametrize("captured", [False, True])
def test_evictions_in_a_row_from_slots_in_order(captured):
    """The first eviction knows positions by their slots and returns them for the next one, whose sinks
    and recent tokens are then those of the sequence, not of the slots."""
    layer, W, rng = make(norms=False, n_seqs=2, width=256)
    lens = [200, 70]
    layer.pool.normal_()
    layer.seq_lens.copy_(i32(lens))
    w = torch.rand((2, 256), device=DEV)
    w[0, :4] = 0                                       # sinks and recent tokens are the lightest
    w[0, 190:200] = 0
    w[1, 60:70] = 0
    W0, pos = w.cpu().numpy().copy(), [list(range(L)) for L in lens]
    cuts = ([120, 50], [40, 20], [30, 19])

    def loop():
        slot_pos, kept = None, []
        for cut in cuts:
            slot_pos = layer.evict(w, budgets[str(cut)], 4, 10, slot_pos)
            kept.append((slot_pos.clone(), w.clone(), layer.seq_lens.clone()))
        return kept
    budgets = {str(cut): i32(cut) for cut in cuts}
    if captured:
        state = [t.clone() for t in (layer.pool, layer.seq_lens, w)]
        loop()                                         # allocates
        side = torch.cuda.Stream()
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=side):
            kept = loop()
        for t, s in zip((layer.pool, layer.seq_lens, w), state):
            t.copy_(s)
        g.replay()
    else:
        kept = loop()
    assert status() == 0
    held = [W0[b, :L] for b, L in enumerate(lens)]
    for cut, (sp, ww, ll) in zip(cuts, kept):
        for b in range(2):
            pairs, new = oracle.evict(held[b], pos[b], cut[b], 4, 10)
            keep = list(range(new))
            for to, frm in pairs:
                keep[to] = frm
            held[b], pos[b] = held[b][keep], [pos[b][k] for k in keep]
            assert ll[b].item() == new
            np.testing.assert_array_equal(sp[b, :new].cpu().numpy(), pos[b])
            np.testing.assert_array_equal(ww[b, :new].cpu().numpy(), held[b])
            assert set(range(4)) | set(range(lens[b] - 10, lens[b])) <= set(pos[b])


@gpu
def test_eviction_updates_the_positions_it_is_given():
    layer, W, rng = make(norms=False, n_seqs=1, width=128)
    layer.pool.normal_()
    layer.seq_lens.fill_(100)
    sp = torch.arange(128, dtype=torch.int32, device=DEV)[None].contiguous()
    out = layer.evict(torch.rand((1, 128), device=DEV), i32([60]), 2, 5, sp)
    assert out is sp and status() == 0 and len(set(sp[0, :60].tolist())) == 60


def _evicted(n_seqs, seed, norms=True):
    """A layer whose caches were cut, its reference, and what a loop then knows: cached tokens and next
    positions of every sequence."""
    layer, W, rng = make(norms=norms, n_seqs=n_seqs, seed=seed)
    d, ctx, cut = layer.dims, [150, 70, 64][:n_seqs], [90, 70, 31][:n_seqs]
    h_ctx = [q(rng.standard_normal((k, d.d_model)), "bf16") for k in ctx]
    layer.prefill_from_hidden(h_ctx)
    layer.seq_lens.copy_(i32(ctx))
    ref = Reference(d, W, n_seqs)
    w = torch.rand((n_seqs, 512), device=DEV)
    held = w.cpu().numpy()
    sp = layer.evict(w, i32(cut), 2, 5)
    for b in range(n_seqs):
        rows = ref.new_rows(h_ctx[b], np.arange(ctx[b]))[1]
        pairs, new = oracle.evict(held[b, :ctx[b]], list(range(ctx[b])), cut[b], 2, 5)
        assert new == cut[b]
        keep = list(range(new))
        for to, frm in pairs:
            keep[to] = frm
        ref.rows[b] = rows[keep]
    assert status() == 0
    return layer, ref, rng, cut, ctx, sp


TOL = dict(max_abs=6e-2, mean_abs=6e-3, rel_l2=2e-2)       # as for the loop of test_gpu_serving


@gpu
@pytest.mark.parametrize("norms", [True, False])
def test_prefill_chunk_behind_an_eviction(norms):
    layer, ref, rng, cut, ctx, _ = _evicted(1, 21, norms)
    T = 100
    h, bi, pos, places = tokens(rng, layer, [T], ctx, cut)
    before = layer.pool.clone()
    bf = layer.prefill_chunk(to_dev(h, "bf16"), i32(pos), i32(bi), 0, T, cut[0] + T, places=i32(places))
    assert status() == 0
    out, _, lse, _ = ref.extend(h, [0, T], pos)
    check(to_np(bf["out"]), out, "bf16", "out", TOL)
    check(to_np(bf["lse"]), lse, "bf16", "lse", dict(max_abs=6e-2, mean_abs=6e-3))
    table = layer.page_table[0].cpu().numpy()
    a, z = bits(before), bits(layer.pool)
    changed = [s for s in range(512) if (a[table[s // 64], s % 64] != z[table[s // 64], s % 64]).any()]
    assert changed == list(range(cut[0], cut[0] + T))


@gpu
def test_pipelines_behind_an_eviction():
    n = 3
    layer, ref, rng, cut, ctx, _ = _evicted(n, 22)
    pipe = DecodePipeline(layer, n, 1, placed=True)
    outs, want = [], []
    pin = lambda x, t: torch.from_numpy(np.asarray(x)).to(t).pin_memory()  # noqa: E731
    lens, nxt = list(cut), list(ctx)
    start = layer.pool.clone()
    steps = [tokens(rng, layer, [1] * n, [p + k for p in nxt], [L + k for L in lens]) for k in range(3)]
    for k, (h, bi, pos, places) in enumerate(steps):
        pipe.wait()
        layer.seq_lens.copy_(i32([L + k + 1 for L in lens]))
        out = torch.empty((n, 256)).pin_memory()
        pipe.submit(pin(h, torch.bfloat16), pin(bi, torch.int32), pin(pos, torch.int32), out,
                    pin(places, torch.int32))
        outs.append(out)
        want.append(ref.extend(h, np.arange(n + 1), pos)[0])
    pipe.wait()
    assert status() == 0
    for got, w in zip(outs, want):
        check(got.numpy(), w, "bf16", "out", TOL)
    with pytest.raises(ValueError):
        pipe.submit(None, None, None, None)
    with pytest.raises(ValueError):
        DecodePipeline(layer, n, 1).submit(None, None, None, None, torch.zeros(n, dtype=torch.int32))
    # the same tokens as one chunk of the first sequence, through the prefill pipeline
    layer.pool.copy_(start)
    h = np.concatenate([s[0][:1] for s in steps])
    pos, places, zero = np.arange(3) + ctx[0], np.arange(3) + cut[0], np.zeros(3)
    pipe = PrefillPipeline(layer, 0, 3, cut[0] + 3)
    out = torch.empty((3, 256), dtype=torch.bfloat16).pin_memory()
    pipe.submit(pin(h, torch.bfloat16), pin(zero, torch.int32), pin(pos, torch.int32), out,
                pin(places, torch.int32))
    pipe.wait()
    assert status() == 0
    check(out.float().numpy(), np.stack([w[0] for w in want]), "bf16", "out", TOL)


@gpu
def test_a_longest_chunk_above_the_tokens_there_are():
    """max_q bounds the chunks of every step a program makes; a step may have fewer tokens than that."""
    layer, W, rng = make(norms=False, n_seqs=2)
    ctx = [30, 100]
    layer.prefill_from_hidden([q(rng.standard_normal((k, 256)), "bf16") for k in ctx])
    h, bi, pos, _ = tokens(rng, layer, [1, 2], ctx, ctx)
    layer.seq_lens.copy_(i32([31, 102]))
    args = (to_dev(h, "bf16"), i32(bi), i32(pos), i32([0, 1, 3]), 3)
    got = []
    for max_q in (2, 64):
        bf = layer.extend(*args, max_q)
        w = torch.zeros((2, 128), device=DEV)
        layer.gather_weights(bf, args[3], 3, max_q, w)
        got.append([bf["out"].clone(), w])
    assert status() == 0
    assert torch.equal(got[0][0], got[1][0]) and torch.equal(got[0][1], got[1][1])
    layer.extend(args[0][:0], args[1], args[2], args[3] * 0, 0, 64)
    assert status() == 0
