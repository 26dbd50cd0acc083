"""mla_chunk_attention against attention in 64 bits, and its refusals.

Tolerance, row by row, with p and v of the fp64 reference, A = sum_t p_t |v_t| and u = 2^-8 (half a
step of bf16).  Scores: 36 MMA steps of 16 products accumulate in fp32, so a score is off by at
most 36 * 2^-23 * scale * sum_e |q_e k_e| =: d (2^-23: the accumulator may round toward zero);
ex2, the scaling and the sums add less than 2^-19.  So p is off by a factor within 1 +- 2 (d +
2^-19), and by one rounding to bf16, and o by one more rounding:
    |o - ref| <= u |ref| + (u + 2 (d + 2^-19)) (1 + u) A + (tokens / 16) 2^-23 A
(the last term: accumulation of the value product).  lse: d + 2^-19 + 2^-22 |lse|.
"""

import ctypes

import numpy as np
import pytest
import torch

from mla_latent_kv_35_b200 import binding as B
from gpu_util import dims, ensure_lib, status
from serving_util import DEV, bits, i32, paged

gpu = pytest.mark.gpu
U = 2.0 ** -8


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if torch.cuda.is_available():
        ensure_lib()
        B.mla_get_device_status()


def workspace(d, nB, total, max_q):
    return torch.full((B.mla_chunk_attention_workspace_size(d, nB, total, max_q),), 0xFF,
                      dtype=torch.uint8, device=DEV)


def call(d, q, cu, total, max_q, pool, n_pages, table, lens, ws=None):
    nB, H = len(lens), d.n_heads
    o = torch.full((total, H, 512), 5.0, dtype=torch.bfloat16, device=DEV)
    lse = torch.full((total, H), 5.0, device=DEV)
    B.mla_chunk_attention(d, q, cu, total, max_q, pool, n_pages, table, table.shape[1], lens, nB,
                          workspace(d, nB, total, max_q) if ws is None else ws, o, lse)
    return o, lse


def reference(q, rows, j, T, scale):
    """(o, lse, A, d) of query j of T over one sequence's rows, all heads, in 64 bits."""
    see = len(rows) - T + j + 1
    k = torch.from_numpy(rows[:see]).to(DEV)
    x = q.double()
    s = x @ k.T * scale
    p = torch.softmax(s, 1)
    d = 36 * 2.0 ** -23 * scale * (x.abs() @ k.abs().T).amax(1)
    return p @ k[:, :512], torch.logsumexp(s, 1), p @ k[:, :512].abs(), d


def check_rows(o, lse, q, rows, T, scale, which=None):
    for j in (range(T) if which is None else which):
        ref, rl, A, d = reference(q[j], rows, j, T, scale)
        e = 2 * (d + 2.0 ** -19)[:, None]
        tol = U * ref.abs() + (U + e) * (1 + U) * A + len(rows) / 16 * 2.0 ** -23 * A
        err = (o[j].double() - ref).abs()
        assert (err <= tol).all(), (j, err.max().item(), (err / tol).max().item())
        le = (lse[j].double() - rl).abs()
        assert (le <= d + 2.0 ** -19 + 2.0 ** -22 * rl.abs()).all(), (j, le.max().item())
        # typical errors are far below the bound: the roundings are independent
        rel = (o[j].double() - ref).norm() / ref.norm()
        assert rel <= 1e-2, rel.item()


def run(H, qs, lens, seed=0, spare=0, peak=1.0, extra=0, which=None):
    rng = np.random.default_rng(seed)
    d = dims("bf16", H=H)
    pool, table, n_pages, rows = paged(rng, lens, 576, torch.bfloat16, extra=extra)
    total = sum(qs) + spare
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    q = (peak * torch.randn((total, H, 576), generator=g, device=DEV)).bfloat16()
    cu = np.concatenate([[0], np.cumsum(qs)])
    o, lse = call(d, q, i32(cu), total, max(max(qs), 1), pool, n_pages, table, i32(lens))
    assert status() == 0
    for b, (T, L) in enumerate(zip(qs, lens)):
        a = slice(cu[b], cu[b + 1])
        check_rows(o[a], lse[a], q[a], rows[b], T, d.scale, None if which is None else which(T))
    assert (o[cu[-1]:] == 5).all() and (lse[cu[-1]:] == 5).all()
    return o, lse


@gpu
@pytest.mark.parametrize("H", [1, 3, 16, 64, 128, 160])
@pytest.mark.parametrize("qs,lens", [
    ([1], [1]), ([1], [300]), ([3], [3]), ([5], [70]), ([2, 2], [2, 513]),
    ([0, 5, 1, 33, 0, 17], [10, 255, 256, 257, 0, 1000]),
])
def test_ragged(H, qs, lens):
    run(H, qs, lens, seed=H, spare=3, extra=H % 2)


@gpu
@pytest.mark.parametrize("L", [63, 64, 65, 127, 128, 255, 256, 257, 511, 512, 513, 769])
def test_edges_of_pages_and_blocks(L):
    run(16, [11], [L], seed=L)
    run(128, [2, 1], [L, L + 1], seed=L)


@gpu
@pytest.mark.parametrize("H,T,L", [(128, 130, 700), (16, 257, 257), (8, 600, 5000), (128, 64, 9000)])
def test_long_chunks(H, T, L):
    run(H, [T], [L], seed=T, which=lambda T: sorted({0, 1, T // 3, T // 2, T - 2, T - 1}))


@gpu
def test_more_workers_than_blocks_and_many_sequences():
    rng = np.random.default_rng(1)
    run(32, [1] * 150, [int(x) for x in rng.integers(1, 400, 150)], seed=2)
    run(16, [int(x) for x in rng.integers(0, 9, 1100)], [int(x) for x in rng.integers(9, 90, 1100)],
        seed=3, which=lambda T: [T - 1] if T else [])


@gpu
def test_no_queries():
    """Room for tokens, but no chunk brings any."""
    d = dims("bf16", H=16)
    pool, table, n_pages, _ = paged(np.random.default_rng(0), [70, 300], 576, torch.bfloat16)
    q = torch.randn((5, 16, 576), device=DEV).bfloat16()
    o, lse = call(d, q, i32([0, 0, 0]), 5, 3, pool, n_pages, table, i32([70, 300]))
    assert status() == 0
    assert (o == 5).all() and (lse == 5).all()


@gpu
def test_many_short_row_blocks_behind_a_long_one():
    """Row blocks of one token block each, next to one of many: splits fall on row blocks' starts."""
    run(128, [1, 40, 1], [20000, 40, 700], seed=11, which=lambda T: sorted({0, T // 2, T - 1}))
    run(16, [7, 200, 64, 1], [12000, 200, 64, 1], seed=12, which=lambda T: sorted({0, T // 2, T - 1}))


@gpu
def test_peaked_scores():
    run(16, [9, 1], [600, 2000], seed=4, peak=6.0)


@gpu
def test_decode_is_a_chunk_of_one_or_two():
    rng = np.random.default_rng(5)
    lens, H = [700, 64, 3000], 128
    d = dims("bf16", H=H)
    pool, table, n_pages, rows = paged(rng, lens, 576, torch.bfloat16)
    for S_q in (1, 2):
        q = torch.randn((3 * S_q, H, 576), device=DEV).bfloat16()
        o, lse = call(d, q, i32(np.arange(4) * S_q), 3 * S_q, S_q, pool, n_pages, table, i32(lens))
        o2 = torch.empty((3, S_q, H, 512), device=DEV)
        l2 = torch.empty((3, S_q, H), device=DEV)
        ws = torch.empty(B.mla_decode_workspace_size(d, 3, S_q), dtype=torch.uint8, device=DEV)
        B.mla_decode(d, q, pool, n_pages, table, table.shape[1], i32(lens), 3, S_q, 0, ws, o2, l2)
        assert status() == 0
        # the same products, split at other blocks: a P rounded on either side of a rescale
        A = 4.0                                       # |v| of N(0, 1) rows averages below this
        assert (o.float() - o2.view(o.shape)).abs().max() <= U * o2.abs().max() + 2 * U * A
        assert (lse - l2.view(lse.shape)).abs().max() <= 2.0 ** -17


@gpu
def test_same_bits_again_on_another_stream_and_in_a_graph():
    rng = np.random.default_rng(6)
    H, qs, lens = 64, [3, 40], [900, 2500]
    d = dims("bf16", H=H)
    pool, table, n_pages, rows = paged(rng, lens, 576, torch.bfloat16)
    q = torch.randn((43, H, 576), device=DEV).bfloat16()
    cu, ld = i32([0, 3, 43]), i32(lens)
    o, lse = call(d, q, cu, 43, 40, pool, n_pages, table, ld)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        o2, lse2 = call(d, q, cu, 43, 40, pool, n_pages, table, ld)
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(o, o2) and torch.equal(lse, lse2)
    ws = workspace(d, 2, 43, 40)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        o3, lse3 = call(d, q, cu, 43, 40, pool, n_pages, table, ld, ws)
    ld.copy_(i32([800, 64]))                           # a replay reads the lengths of its time
    cu.copy_(i32([0, 7, 40]))
    g.replay()
    o4, lse4 = call(d, q, cu, 43, 40, pool, n_pages, table, ld)
    assert torch.equal(o3, o4) and torch.equal(lse3, lse4) and not torch.equal(o3, o)
    assert status() == 0
    check_rows(o4[7:40], lse4[7:40], q[7:40], rows[1][:64], 33, d.scale)


def _bad(lens, qs, cu, total, max_q, table=None, n_pages=None, seed=7, H=16):
    rng = np.random.default_rng(seed)
    d = dims("bf16", H=H)
    pool, t, n, rows = paged(rng, [min(max(L, 1), 300) for L in lens], 576, torch.bfloat16, unused=0.0)
    q = torch.randn((total, H, 576), device=DEV).bfloat16()
    if table is not None:
        t = table(t)
    o, lse = call(d, q, i32(cu), total, max_q, pool, n if n_pages is None else n_pages, t, i32(lens))
    assert status() == 5
    return d, q, rows, o, lse


@gpu
@pytest.mark.parametrize("bad", [-1, 3, 100000])       # negative, fewer than its queries, past the table
def test_bad_lengths_see_nothing(bad):
    d, q, rows, o, lse = _bad([200, bad, 90], None, [0, 2, 6, 9], 9, 4)
    assert (o[2:6] == 0).all() and (lse[2:6] == -float("inf")).all()
    check_rows(o[:2], lse[:2], q[:2], rows[0], 2, d.scale)
    check_rows(o[6:9], lse[6:9], q[6:9], rows[2], 3, d.scale)


@gpu
@pytest.mark.parametrize("cu,max_q", [([0, 2, 1, 5], 4), ([0, 2, 7, 99], 5), ([-3, 2, 4, 5], 4),
                                      ([0, 2, 8, 9], 5)])
def test_bad_chunks_leave_every_row(cu, max_q):
    d, q, rows, o, lse = _bad([200, 300, 90], None, cu, 9, max_q)
    assert (o == 5).all() and (lse == 5).all()


@gpu
def test_bad_pages_count_as_zero_rows():
    def table(t):
        t = t.clone()
        t[0, 1], t[1, 0] = -1, 1000
        return t
    d, q, rows, o, lse = _bad([200, 60], None, [0, 2, 4], 4, 2, table)
    rows[0][64:128] = 0
    rows[1][:] = 0
    check_rows(o[:2], lse[:2], q[:2], rows[0], 2, d.scale)
    assert (o[2:4] == 0).all()


def test_refused_on_the_host():
    from mla_latent_kv_35_b200 import build
    build.build()
    lib = B.lib()
    x = 1 << 12

    def f(d=dims("bf16"), q=x, cu=x, total=8, max_q=4, pool=x, n_pages=4, pt=x, mp=2, sl=x, nB=2, ws=x,
          wb=1 << 40, o=x, lse=x):
        return lib.mla_chunk_attention(ctypes.byref(d.c()), q, cu, total, max_q, pool, n_pages, pt, mp, sl,
                                       nB, ws, wb, o, lse, 0)
    assert f(nB=0, q=0) == 0 and f(total=0, max_q=0, q=0) == 0
    for kw in (dict(q=0), dict(cu=0), dict(pool=0), dict(pt=0), dict(sl=0), dict(ws=0), dict(o=0), dict(lse=0),
               dict(q=x + 2), dict(pool=x + 8), dict(o=x + 4), dict(ws=x + 128), dict(wb=1000), dict(nB=-1),
               dict(total=-1), dict(max_q=-1), dict(max_q=9), dict(n_pages=0), dict(mp=0),
               dict(total=1 << 24), dict(mp=1 << 30),
               dict(mp=(1 << 25) - 1), dict(total=1 << 23, mp=1024)):
        assert f(**kw) == 1, kw
    for d in (dims("f32"), dims("bf16", dc=256), dims("bf16", dr=32), dims("bf16", page=32)):
        assert f(d=d) == 2
        assert B.mla_chunk_attention_workspace_size(d, 2, 8, 4) == 0
    assert B.mla_chunk_attention_workspace_size(dims("bf16"), 2, 1 << 24, 4) == 0
    a, b = (B.mla_chunk_attention_workspace_size(dims("bf16"), 2, n, 4) for n in (8, 4096))
    assert 0 < a < b


@gpu
def test_binding_refuses_wrong_tensors():
    rng = np.random.default_rng(8)
    d = dims("bf16", H=4)
    pool, table, n_pages, _ = paged(rng, [70, 80], 576, torch.bfloat16)
    good = dict(q=torch.zeros((3, 4, 576), dtype=torch.bfloat16, device=DEV), cu=i32([0, 1, 3]), pool=pool,
                table=table, lens=i32([70, 80]), ws=workspace(d, 2, 3, 2),
                o=torch.zeros((3, 4, 512), dtype=torch.bfloat16, device=DEV), lse=torch.zeros((3, 4), device=DEV))

    def f(**kw):
        a = {**good, **kw}
        B.mla_chunk_attention(d, a["q"], a["cu"], 3, 2, a["pool"], n_pages, a["table"], table.shape[1],
                              a["lens"], 2, a["ws"], a["o"], a["lse"])
    f()
    for kw in (dict(q=good["q"].float()), dict(q=good["q"][:2]), dict(q=good["q"].cpu()),
               dict(q=good["q"].transpose(0, 1)), dict(cu=good["cu"][:2]), dict(cu=good["cu"].long()),
               dict(pool=pool[:1]), dict(table=table[:1]), dict(lens=good["lens"][:1]),
               dict(o=good["o"].float()), dict(o=good["o"][:2]), dict(lse=good["lse"].double())):
        with pytest.raises(ValueError):
            f(**kw)
    with pytest.raises(B.MLAError):
        f(ws=good["ws"][256:])
    assert status() == 0


@gpu
@pytest.mark.parametrize("T", [1, 5, 130])
def test_out_proj_of_bf16_rows_is_out_proj(T):
    d = dims("bf16", H=16, dm=256)
    g = torch.Generator(device=DEV)
    g.manual_seed(T)
    mk = lambda *n: torch.randn(n, generator=g, device=DEV).bfloat16()  # noqa: E731
    o, w_uv, w_o = mk(T, 16, 512), mk(16, 128, 512), mk(256, 16 * 128)
    a, b = torch.empty((T, 256), device=DEV), torch.empty((T, 256), device=DEV)
    s1 = torch.empty(B.mla_out_proj_scratch_size(d, T), dtype=torch.uint8, device=DEV)
    s2 = torch.empty(B.mla_out_proj_bf16_scratch_size(d, T), dtype=torch.uint8, device=DEV)
    B.mla_out_proj(d, o.float(), w_uv, w_o, s1, a, T)
    B.mla_out_proj_bf16(d, o, w_uv, w_o, s2, b, T)
    assert status() == 0
    np.testing.assert_array_equal(bits(a), bits(b))
