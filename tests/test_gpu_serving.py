"""A serving loop through MLADecodeLayer: norms, ragged chunks, gathered attention weights, eviction.

The reference follows the loop in 64 bits from the same hidden states and weights: projection, the
oracle's norms and rotation, its attention over the tokens the cache should hold, W_UV and W_O.  The
choice of what to evict is fed from the GPU's own weights (two tokens may weigh the same to the last
bit), which are checked against the reference's on their own.

Tolerance.  Between hidden state and output stand five roundings to bf16 that the reference does not
make (the A0 row, the normed or rotated row, the absorbed query, P, o_lat), each at most u = 2^-8 of a
number; rows of unit mean square hold numbers up to about 3: at most 5 * 3 * u = 6e-2, independent and
so far less on average (sqrt(5 / 3) u = 5e-3 of the norm).  A score is a sum of 576 products with
independent relative errors of two such roundings, off by less than 6e-2 at |s| <= 4 (five standard
deviations of u sqrt(2 / 3) |s|); a gathered weight is its exponential, off by that much relative.
"""

import numpy as np
import pytest
import torch

import oracle
from mla_latent_kv_35_b200 import binding as B
from mla_latent_kv_35_b200 import workloads as wl
from mla_latent_kv_35_b200.engine import MLADecodeLayer
from gpu_util import DEV, check, dims, ensure_lib, q, status, to_dev, to_np
from serving_util import i32, page_table

gpu = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if torch.cuda.is_available():
        ensure_lib()
        B.mla_get_device_status()


class Reference:
    """One layer in 64 bits; the cache of each sequence is a list of (row, position)."""

    def __init__(self, d, W, n_seqs):
        self.d, self.W = d, W
        self.rows = [np.zeros((0, d.d_latent + d.d_rope)) for _ in range(n_seqs)]

    def new_rows(self, h, pos):
        d, W = self.d, self.W
        y = oracle.project(h, np.concatenate([W["W_Q"], W["W_DKV"], W["W_KR"]], 0))
        return oracle.norm_rope(y, d.n_heads, d.d_nope, d.d_rope, d.d_latent, W.get("N_Q"), W.get("N_C"),
                                W.get("N_KR"), 1e-6, pos)

    def extend(self, h, cu, pos):
        """(out [T, d_model], o_lat, lse, weights per sequence) of one ragged step."""
        d = self.d
        qs, ckr = self.new_rows(h, pos)
        qa = np.concatenate([np.stack([qs[:, i, :d.d_nope] @ self.W["W_UK"][i].astype(np.float64)
                                       for i in range(d.n_heads)], 1), qs[..., d.d_nope:]], -1)
        o, lse, got = [], [], []
        for b in range(len(cu) - 1):
            a, z = cu[b], cu[b + 1]
            self.rows[b] = np.concatenate([self.rows[b], ckr[a:z]])
            r = self.rows[b]
            if z == a:
                got.append(np.zeros(len(r)))
                continue
            att = oracle.latent_attention(qa[a:z], r[:, :d.d_latent], r[:, d.d_latent:], d.scale)
            o.append(att["o_lat"])
            lse.append(att["lse"])
            got.append(oracle.attention_weights(qa[a:z], r, att["lse"], d.scale))
        o, lse = np.concatenate(o), np.concatenate(lse)
        return oracle.out_proj(o, self.W["W_UV"], self.W["W_O"])[1], o, lse, got


def make(dtype="bf16", norms=True, H=8, dm=256, page=64, kind="bf16", width=512, n_seqs=3, seed=0, **kw):
    d = dims(dtype, H=H, dm=dm, page=page, **kw)
    rng = np.random.default_rng(seed)
    dqk = d.d_nope + d.d_rope
    w = lambda *s: q(rng.standard_normal(s) / np.sqrt(s[-1]), dtype)  # noqa: E731
    W = dict(W_Q=w(H * dqk, dm), W_DKV=w(d.d_latent, dm), W_KR=w(d.d_rope, dm), W_UK=w(H, d.d_nope, d.d_latent),
             W_UV=w(H, d.d_v, d.d_latent), W_O=w(dm, H * d.d_v))
    if norms:
        n = lambda k: q(1 + 0.2 * rng.standard_normal(k), dtype)  # noqa: E731
        W.update(N_Q=n(dqk), N_C=n(d.d_latent), N_KR=n(d.d_rope))
    layer = MLADecodeLayer(d, W, DEV)
    table, n_pages = page_table(rng, [width] * n_seqs, page)
    if kind == "fp8":
        pool = torch.full((n_pages, page, 656), 0xFF, dtype=torch.uint8, device=DEV)
    else:
        pool = torch.full((n_pages, page, d.d_latent + d.d_rope), float("nan"), dtype=d.torch_dtype, device=DEV)
    layer.set_cache(pool, torch.from_numpy(table).to(DEV), torch.zeros(n_seqs, dtype=torch.int32, device=DEV),
                    kind=kind)
    return layer, W, rng


def tokens(rng, layer, qs, next_pos, lens):
    """Hidden states, batch index, positions and places of a ragged step's new tokens."""
    T, dt = sum(qs), layer.dims.dtype
    h = q(rng.standard_normal((T, layer.dims.d_model)), dt)
    bi = np.repeat(np.arange(len(qs)), qs)
    pos = np.concatenate([np.arange(p, p + n) for p, n in zip(next_pos, qs)])
    places = np.concatenate([np.arange(L, L + n) for L, n in zip(lens, qs)])
    return h, bi, pos, places


@gpu
@pytest.mark.parametrize("norms", [True, False])
def test_chunks_weights_and_eviction_in_a_loop(norms):
    layer, W, rng = make(norms=norms)
    d, n = layer.dims, 3
    ref = Reference(d, W, n)
    width = 512
    weights = torch.zeros((n, width), device=DEV)
    slot_pos = torch.zeros((n, width), dtype=torch.int32, device=DEV)
    held, lens, nxt = [np.zeros(0)] * n, [0] * n, [0] * n      # gathered so far, cached, next position
    posn = [[] for _ in range(n)]
    plan = [([130, 7, 64], None), ([1, 1, 1], [100, 8, 50]), ([5, 0, 33], None), ([2, 130, 1], [90, 90, 40]),
            ([1, 1, 1], [80, 91, 41]), ([4, 3, 1], None)]
    for qs, budget in plan:
        h, bi, pos, places = tokens(rng, layer, qs, nxt, lens)
        T, cu = sum(qs), np.concatenate([[0], np.cumsum(qs)])
        layer.seq_lens.copy_(i32([L + k for L, k in zip(lens, qs)]))
        bf = layer.extend(to_dev(h, "bf16"), i32(bi), i32(pos), i32(cu), T, max(qs), places=i32(places))
        layer.gather_weights(bf, i32(cu), T, max(qs), weights)
        assert status() == 0
        out, o, lse, got = ref.extend(h, cu, pos)
        check(to_np(bf["o_lat"]), o, "bf16", "o_lat", dict(max_abs=6e-2, mean_abs=6e-3, rel_l2=2e-2))
        check(to_np(bf["lse"]), lse, "bf16", "lse", dict(max_abs=6e-2, mean_abs=6e-3))
        check(to_np(bf["out"]), out, "bf16", "out", dict(max_abs=6e-2, mean_abs=6e-3, rel_l2=2e-2))
        for b in range(n):
            lens[b] += qs[b]
            posn[b] += list(range(nxt[b], nxt[b] + qs[b]))
            nxt[b] += qs[b]
            slot_pos[b, lens[b] - qs[b]:lens[b]] = i32(posn[b][lens[b] - qs[b]:])
            held[b] = np.concatenate([held[b], np.zeros(qs[b])]) + got[b]
            mine = to_np(weights[b, :lens[b]])
            # a weight is exp of a score: relative errors are the score's absolute ones
            np.testing.assert_allclose(mine, held[b], rtol=6e-2, atol=6e-2 * max(1e-3, held[b].mean()))
        if budget is not None:
            before = weights.clone()
            layer.evict(weights, i32(budget), 2, 3, slot_pos)
            assert status() == 0
            for b in range(n):
                pairs, new = oracle.evict(before[b, :lens[b]].cpu().numpy(), posn[b], budget[b], 2, 3)
                keep = list(range(new))
                for to, frm in pairs:
                    keep[to] = frm
                ref.rows[b] = ref.rows[b][keep]
                held[b] = to_np(before[b, :lens[b]])[keep]
                posn[b] = [posn[b][k] for k in keep]
                lens[b] = new
                np.testing.assert_array_equal(slot_pos[b, :new].cpu().numpy(), posn[b])
                np.testing.assert_array_equal(to_np(weights[b, :new]), held[b])
            assert layer.seq_lens.tolist() == lens
            # entries behind the new end are stale; the loop's own slots start from nothing
            for b in range(n):
                weights[b, lens[b]:] = 0


@gpu
@pytest.mark.parametrize("dtype,kind", [("bf16", "bf16"), ("bf16", "fp8"), ("f32", "bf16")])
def test_decode_steps_of_a_normed_layer(dtype, kind):
    """step() of a layer with norms, after prefill_from_hidden, for every cache kind."""
    kw = dict(dn=32, dc=64, dr=16) if dtype == "f32" else {}
    layer, W, rng = make(dtype, True, kind=kind, **kw)
    d, n = layer.dims, 3
    ctx = [70, 1, 129]
    h_ctx = [q(rng.standard_normal((k, d.d_model)), dtype) for k in ctx]
    layer.prefill_from_hidden(h_ctx)
    ref = Reference(d, W, n)
    for b in range(n):
        ref.rows[b] = ref.new_rows(h_ctx[b], np.arange(ctx[b]))[1]
    for S_q in (1, 2):
        h, bi, pos, _ = tokens(rng, layer, [S_q] * n, ctx, ctx)
        ctx = [c + S_q for c in ctx]
        layer.seq_lens.copy_(i32(ctx))
        bf = layer.step(to_dev(h, dtype), i32(bi), i32(pos), n, S_q)
        assert status() == 0
        out, o, lse, _ = ref.extend(h, np.arange(n + 1) * S_q, pos)
        # the bf16 cache rows, queries and P; the 8-bit cache adds 2^-4 of each latent number
        tol = None if dtype == "f32" else dict(max_abs=6e-2, mean_abs=6e-3, rel_l2=2e-2) if kind == "bf16" else \
            dict(max_abs=0.25, mean_abs=3e-2, rel_l2=6e-2)
        check(to_np(bf["o_lat"]).reshape(o.shape), o, dtype, "o_lat", tol)
        check(to_np(bf["out"]), out, dtype, "out", tol)


@gpu
def test_prefill_chunk_of_a_normed_layer():
    layer, W, rng = make(n_seqs=1)
    d, T, L0 = layer.dims, 200, 60
    h_ctx = q(rng.standard_normal((L0, d.d_model)), "bf16")
    layer.prefill_from_hidden([h_ctx])
    ref = Reference(d, W, 1)
    ref.rows[0] = ref.new_rows(h_ctx, np.arange(L0))[1]
    h, bi, pos, _ = tokens(rng, layer, [T], [L0], [L0])
    bf = layer.prefill_chunk(to_dev(h, "bf16"), i32(pos), i32(bi), 0, T, L0 + T)
    assert status() == 0
    out, _, lse, _ = ref.extend(h, [0, T], pos)
    check(to_np(bf["out"]), out, "bf16", "out", dict(max_abs=6e-2, mean_abs=6e-3, rel_l2=2e-2))
    check(to_np(bf["lse"]), lse, "bf16", "lse", dict(max_abs=6e-2, mean_abs=6e-3))


@gpu
def test_extend_equals_step_and_places_equal_positions():
    """One token per sequence through extend() and step(), fused or not, with explicit places."""
    layer, W, rng = make(norms=False)
    n, ctx = 3, [100, 3, 64]
    layer.prefill_from_hidden([q(rng.standard_normal((k, 256)), "bf16") for k in ctx])
    h, bi, pos, places = tokens(rng, layer, [1] * n, ctx, ctx)
    layer.seq_lens.copy_(i32([c + 1 for c in ctx]))
    hd = to_dev(h, "bf16")
    pool = layer.pool.clone()
    a = {k: v.clone() for k, v in layer.step(hd, i32(bi), i32(pos), n, 1).items()}
    appended = layer.pool.clone()
    outs = []
    for fused, pl in ((True, None), (False, None), (True, i32(places))):
        layer.pool.copy_(pool)
        bf = layer.extend(hd, i32(bi), i32(pos), i32([0, 1, 2, 3]), 3, 1, fused=fused, places=pl)
        assert status() == 0
        assert torch.equal(layer.pool.view(torch.int16), appended.view(torch.int16))
        assert torch.equal(bf["qbuf"].view(torch.int16), a["qbuf"].view(torch.int16))
        outs.append(bf["out"].clone())
    assert torch.equal(outs[0], outs[1]) and torch.equal(outs[0], outs[2])
    check(to_np(outs[0]), to_np(a["out"]), "bf16", "out")


@gpu
def test_a_graph_of_a_step_with_its_weights_and_eviction():
    """The whole decode step, the gathering and an eviction captured once and replayed: every replay
    appends at the place and position the host wrote, and leaves every sequence at its budget."""
    layer, W, rng = make(norms=True, n_seqs=2, seed=3)
    n, budget = 2, [40, 60]
    ctx = [40, 60]
    layer.prefill_from_hidden([q(rng.standard_normal((k, 256)), "bf16") for k in ctx])
    weights = torch.zeros((n, 512), device=DEV)
    slot_pos = torch.zeros((n, 512), dtype=torch.int32, device=DEV)
    for b in range(n):
        slot_pos[b, :ctx[b]] = i32(np.arange(ctx[b]))
    hd = torch.zeros((n, 256), dtype=torch.bfloat16, device=DEV)
    bi, pos, places, cu, bud = i32([0, 1]), i32([0, 0]), i32([0, 0]), i32([0, 1, 2]), i32(budget)
    rows = torch.arange(n, device=DEV)

    def one():
        # places: behind what is cached; the new token's position joins slot_pos
        places.copy_(layer.seq_lens)
        slot_pos[rows, places.long()] = pos
        layer.seq_lens.add_(1)
        bf = layer.step(hd, bi, pos, n, 1, places=places)
        layer.gather_weights(bf, cu, n, 1, weights)
        layer.evict(weights, bud, 1, 4, slot_pos)
        return bf

    layer.seq_lens.copy_(i32(ctx))
    state = [t.clone() for t in (layer.pool, layer.seq_lens, weights, slot_pos)]
    hs = [to_dev(rng.standard_normal((n, 256)).astype(np.float32), "bf16") for _ in range(6)]

    def restore():
        for t, s in zip((layer.pool, layer.seq_lens, weights, slot_pos), state):
            t.copy_(s)
    eager = []
    for k, h in enumerate(hs):
        hd.copy_(h)
        pos.copy_(i32([ctx[0] + k, ctx[1] + k]))
        eager.append(one()["out"].clone())
    assert status() == 0
    after = [t.clone() for t in (layer.seq_lens, weights, slot_pos)]
    assert after[0].tolist() == budget
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=side):
        bf = one()
    restore()
    for k, h in enumerate(hs):
        hd.copy_(h)
        pos.copy_(i32([ctx[0] + k, ctx[1] + k]))
        g.replay()
        assert torch.equal(bf["out"], eager[k])
    assert status() == 0
    for t, s in zip((layer.seq_lens, weights, slot_pos), after):
        assert torch.equal(t, s)
    # sinks and recents are still there
    for b in range(n):
        kept = set(slot_pos[b, :budget[b]].tolist())
        assert {0} | {ctx[b] + k for k in range(2, 6)} <= kept


@gpu
def test_a_graph_of_padded_chunks_and_buffers_of_many_lengths():
    """One captured extend of 9 rows replays with the chunks that cu_q then holds (rows behind them
    pad), as the eager call of just those rows; and steps of other lengths use few sets of buffers."""
    T, n = 9, 3
    layer, W, rng = make(norms=True, n_seqs=n, seed=5)
    ctx = [30, 1, 200]
    h_ctx = [q(rng.standard_normal((k, 256)), "bf16") for k in ctx]
    layer.prefill_from_hidden(h_ctx)
    ref = Reference(layer.dims, W, n)
    rows = [ref.new_rows(x, np.arange(k))[1] for x, k in zip(h_ctx, ctx)]
    start = layer.pool.clone()
    spare = 500                                            # a slot that no sequence reaches
    hd = torch.zeros((T, 256), dtype=torch.bfloat16, device=DEV)
    bi, pos, places, cu = i32([0] * T), i32([0] * T), i32([spare] * T), i32([0] * (n + 1))
    layer.extend(hd, bi, pos, cu, T, 5, places=places)     # allocates
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=side):
        bf = layer.extend(hd, bi, pos, cu, T, 5, places=places)
    for qs in ([5, 1, 3], [0, 0, 1], [2, 5, 0], [0, 0, 0], [1, 1, 1]):
        k = sum(qs)
        cum = np.concatenate([[0], np.cumsum(qs)])
        p = np.concatenate([np.arange(c, c + m) for c, m in zip(ctx, qs)] + [np.full(T - k, spare)])
        b = np.concatenate([np.repeat(np.arange(n), qs), np.zeros(T - k)])
        h = q(rng.standard_normal((T, 256)), "bf16")
        layer.seq_lens.copy_(i32(np.array(ctx) + qs))
        layer.pool.copy_(start)
        for t, x in ((hd, to_dev(h, "bf16")), (bi, i32(b)), (pos, i32(p)), (places, i32(p)), (cu, i32(cum))):
            t.copy_(x)
        g.replay()
        got = [bf[name][:k].clone() for name in ("out", "o_lat", "lse")]
        assert status() == 0
        if k == 0:
            continue
        ref.rows = list(rows)
        out, o, lse, _ = ref.extend(h[:k], cum, p[:k])
        for unpadded in (False, True):
            check(to_np(got[1]), o, "bf16", "o_lat", dict(max_abs=6e-2, mean_abs=6e-3, rel_l2=2e-2))
            check(to_np(got[2]), lse, "bf16", "lse", dict(max_abs=6e-2, mean_abs=6e-3))
            check(to_np(got[0]), out, "bf16", "out", dict(max_abs=6e-2, mean_abs=6e-3, rel_l2=2e-2))
            if not unpadded:                               # the same rows alone, in buffers of their own
                layer.pool.copy_(start)
                one = layer.extend(hd[:k], bi[:k], pos[:k], cu, k, 5 if k > 5 else k, places=places[:k], slot=1)
                assert [one[name].shape[0] for name in ("out", "o_lat", "lse", "y", "qbuf")] == [k] * 5
                got = [one[name].clone() for name in ("out", "o_lat", "lse")]
    assert status() == 0
    before = torch.cuda.memory_allocated()
    sets = {key[2] for key in layer._bufs if key[0] == "extend"}
    for k in range(1, 17):
        layer.extend_buffers(n, k, k)
    assert {key[2] for key in layer._bufs if key[0] == "extend"} == sets | {1, 2, 4, 8, 16}
    assert torch.cuda.memory_allocated() - before < 5 * 64 * 2 ** 20
    layer.extend(hd[:0], bi, pos, cu * 0, 0, 0)            # no rows at all
    assert status() == 0


@gpu
def test_two_layers_on_two_streams_at_once():
    """Two layers step, gather and evict on streams of their own at the same time, through graphs and
    eagerly: the same bits as one after the other."""
    n, qs = 3, [70, 1, 5]
    T, cu = sum(qs), np.concatenate([[0], np.cumsum(qs)])
    runs = []
    for seed in (11, 12):
        layer, W, rng = make(norms=True, H=16, n_seqs=n, seed=seed)
        ctx = [200, 64, 129]
        layer.prefill_from_hidden([q(rng.standard_normal((k, 256)), "bf16") for k in ctx])
        h, bi, pos, places = tokens(rng, layer, qs, ctx, ctx)
        lens = i32(np.array(ctx) + qs)
        state = dict(layer=layer, args=(to_dev(h, "bf16"), i32(bi), i32(pos), i32(cu), T, max(qs)),
                     pool=layer.pool.clone(), lens=lens, weights=torch.zeros((n, 512), device=DEV),
                     budget=i32([150, 60, 100]))

        def step(s=state):
            layer = s["layer"]
            layer.pool.copy_(s["pool"])
            layer.seq_lens.copy_(s["lens"])
            s["weights"].zero_()
            bf = layer.extend(*s["args"])
            layer.gather_weights(bf, s["args"][3], T, max(qs), s["weights"])
            layer.evict(s["weights"], s["budget"], 2, 8)
            return [bf["out"], bf["lse"], s["weights"], layer.seq_lens, layer.pool]
        state["step"] = step
        step()
        torch.cuda.synchronize()
        state["ref"] = [t.clone() for t in step()]
        state["stream"] = torch.cuda.Stream()
        state["graph"] = torch.cuda.CUDAGraph()
        torch.cuda.synchronize()
        with torch.cuda.graph(state["graph"], stream=state["stream"]):
            state["outs"] = step()
        runs.append(state)
    assert status() == 0
    torch.cuda.synchronize()
    same = lambda a, b: torch.equal(a.contiguous().view(torch.uint8), b.contiguous().view(torch.uint8))  # noqa: E731
    for eager in (False, True):
        for _ in range(20):
            for s in runs:
                with torch.cuda.stream(s["stream"]):
                    if eager:
                        s["outs"] = s["step"]()
                    else:
                        s["graph"].replay()
        torch.cuda.synchronize()
        assert status() == 0
        for s in runs:
            for a, b in zip(s["outs"], s["ref"]):
                assert same(a, b)


@gpu
def test_refusals_of_the_layer():
    layer, W, rng = make(kind="fp8")
    with pytest.raises(ValueError):
        layer.extend(None, None, None, None, 1, 1)
    with pytest.raises(ValueError):
        layer.gather_weights({}, None, 1, 1, torch.zeros((3, 4), device=DEV))
    layer, W, rng = make("f32", dn=32, dc=64, dr=16)
    with pytest.raises(ValueError):
        layer.extend(None, None, None, None, 1, 1)
