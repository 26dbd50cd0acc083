"""mla_attn_weights against the sums in 64 bits, and its refusals.

Tolerance, per token, with c_r its contributions exp(s - lse) in 64 bits: a score is off by at most
d = 36 * 2^-23 * scale * sum_e |q_e k_e| (36 MMA steps, accumulator may round toward zero), its scaling and
the lse's conversion by 2^-22 (|s scale| + |lse|), ex2 by 2^-21 relative; sums of n rows run in four
chains of at most 32 per group, then the groups: (32 + n / 64 + 4) 2^-24 relative.
"""

import ctypes

import numpy as np
import pytest
import torch

import oracle
from mla_latent_kv_35_b200 import binding as B
from gpu_util import dims, ensure_lib, status
from serving_util import DEV, i32, paged

gpu = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if torch.cuda.is_available():
        ensure_lib()
        B.mla_get_device_status()


def call(d, q, lse, cu, total, max_q, pool, n_pages, table, lens, w_in, keep, w_out):
    B.mla_attn_weights(d, q, lse, cu, total, max_q, pool, n_pages, table, table.shape[1], lens, len(lens),
                       w_in, keep, w_out, w_out.shape[1])


def reference(q, lse, rows, T, scale):
    """(sum, bound of its error) per token, in 64 bits."""
    L, H = len(rows), q.shape[1] if len(q) else 1
    k = torch.from_numpy(rows).to(DEV)
    w = torch.zeros(L, dtype=torch.float64, device=DEV)
    e = torch.zeros_like(w)
    for j in range(T):
        see = L - T + j + 1
        x, l = q[j].double(), lse[j].double()[:, None]
        s = x @ k[:see].T * scale
        ok = l > -float("inf")
        c = torch.where(ok, (s - l).exp(), 0)
        d = 36 * 2.0 ** -23 * scale * (x.abs() @ k[:see].abs().T) + 2.0 ** -22 * (s.abs() + l.abs()) + 2.0 ** -21
        w[:see] += c.sum(0)
        e[:see] += torch.where(ok, c * (2 * d), 0).sum(0)
    n = T * H
    return w, e + (36 + n / 64) * 2.0 ** -24 * w


def run(H, qs, lens, seed=0, keep=1.0, alias=False, with_in=True, pad=3, spare=0, some_inf=False):
    rng = np.random.default_rng(seed)
    d = dims("bf16", H=H)
    pool, table, n_pages, rows = paged(rng, lens, 576, torch.bfloat16, extra=H % 2)
    total = sum(qs) + spare
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    q = torch.randn((total, H, 576), generator=g, device=DEV).bfloat16()
    cu = np.concatenate([[0], np.cumsum(qs)])
    seq = np.repeat(np.arange(len(qs)), qs)
    lse = torch.full((total, H), 3.0, device=DEV)
    if total > spare:
        base = np.log(np.maximum(np.asarray(lens)[seq], 1)) + 1.5
        lse[:len(seq)] = torch.from_numpy(base).float().to(DEV)[:, None] + 0.3 * torch.randn(
            (len(seq), H), generator=g, device=DEV)
    if some_inf:
        lse[::2, ::3] = -float("inf")
    width = max(lens) + pad
    w_in = torch.exp(torch.randn((len(lens), width), generator=g, device=DEV))
    for b, (T, L) in enumerate(zip(qs, lens)):
        w_in[b, max(L - T, 0):] = float("nan") if not alias else 9.0       # not gathered yet
    before = w_in.clone()
    w_out = w_in if alias else torch.full_like(w_in, 9.0)
    call(d, q, lse, i32(cu), total, max(qs), pool, n_pages, table, i32(lens), w_in if with_in else None, keep,
         w_out)
    assert status() == 0
    for b, (T, L) in enumerate(zip(qs, lens)):
        a = slice(cu[b], cu[b + 1])
        ref, tol = reference(q[a], lse[a], rows[b], T, d.scale)
        if with_in and keep != 0:
            ref[:L - T] += keep * before[b, :L - T].double()
        err = (w_out[b, :L].double() - ref).abs()
        tol = tol + 2.0 ** -23 * ref.abs() + 1e-37
        assert (err <= tol).all(), (b, err.max().item(), (err / tol).max().item())
        assert (w_out[b, L:] == 9).all()
    if not alias:
        assert torch.equal(torch.nan_to_num(w_in, nan=-1.0), torch.nan_to_num(before, nan=-1.0))
    return w_out


@gpu
@pytest.mark.parametrize("H", [1, 3, 16, 64, 128])
@pytest.mark.parametrize("qs,lens", [
    ([1], [1]), ([1], [300]), ([1, 1, 1], [64, 1, 1000]), ([2, 2], [2, 513]), ([0, 1, 0], [10, 256, 0]),
    ([3], [3]), ([5], [70]), ([0, 5, 1, 33, 0, 17], [10, 255, 256, 257, 0, 1000]),
])
def test_ragged(H, qs, lens):
    run(H, qs, lens, seed=H)


@gpu
@pytest.mark.parametrize("L", [63, 64, 65, 127, 128, 129, 255, 256, 257, 511, 513])
@pytest.mark.parametrize("H,T", [(128, 1), (128, 2), (16, 30)])
def test_edges_of_pages_and_tiles(H, T, L):
    run(H, [T, 1], [L, L + 1], seed=L)


@gpu
@pytest.mark.parametrize("H,qs", [(16, [1, 3, 0]), (128, [2, 1, 0]), (128, [7, 1, 0])])
@pytest.mark.parametrize("kw", [dict(keep=0.0), dict(keep=0.5), dict(keep=-2.0), dict(with_in=False),
                                dict(alias=True), dict(alias=True, keep=0.9), dict(some_inf=True),
                                dict(spare=2)])
def test_what_is_kept(H, qs, kw):
    run(H, qs, [400, 90, 70], seed=2, **kw)


@gpu
def test_many_sequences():
    rng = np.random.default_rng(1)
    run(16, [1] * 500, [int(x) for x in rng.integers(1, 700, 500)], seed=3)
    run(16, [int(x) for x in rng.integers(0, 40, 450)], [int(x) for x in rng.integers(40, 600, 450)], seed=4)


@gpu
@pytest.mark.parametrize("H,qs,lens", [(128, [1], [70001]), (64, [2, 1], [9000, 33000]), (128, [33], [9001]),
                                       (8, [500], [20000])])
def test_long(H, qs, lens):
    run(H, qs, lens, seed=5)


@gpu
@pytest.mark.parametrize("H,T", [(16, 1), (16, 7), (128, 2), (128, 5)])
def test_after_the_attention_every_row_has_given_one(H, T):
    rng = np.random.default_rng(6)
    lens, d = [700, 64, 3000], dims("bf16", H=H)
    pool, table, n_pages, rows = paged(rng, lens, 576, torch.bfloat16)
    q = torch.randn((3 * T, H, 576), device=DEV).bfloat16()
    cu = i32(np.arange(4) * T)
    o = torch.empty((3 * T, H, 512), dtype=torch.bfloat16, device=DEV)
    lse = torch.empty((3 * T, H), device=DEV)
    ws = torch.empty(B.mla_chunk_attention_workspace_size(d, 3, 3 * T, T), dtype=torch.uint8, device=DEV)
    B.mla_chunk_attention(d, q, cu, 3 * T, T, pool, n_pages, table, table.shape[1], i32(lens), 3, ws, o, lse)
    w = torch.zeros((3, 3000), device=DEV)
    call(d, q, lse, cu, 3 * T, T, pool, n_pages, table, i32(lens), None, 1.0, w)
    assert status() == 0
    # both kernels form the same fp32 scores; what remains is two ex2 and two sums, 2^-17 with room
    assert ((w.double().sum(1) - T * H).abs() <= 2.0 ** -17 * T * H).all(), w.double().sum(1) / (T * H)
    # the sums agree with the oracle's, token by token, for one sequence
    got = oracle.attention_weights(q[T:2 * T].double().cpu().numpy(), rows[1], lse[T:2 * T].double().cpu().numpy(),
                                   d.scale)
    np.testing.assert_allclose(w[1, :64].double().cpu().numpy(), got, rtol=1e-4, atol=1e-7)


@gpu
def test_same_bits_again_on_another_stream_and_in_a_graph():
    rng = np.random.default_rng(7)
    for H, qs in ((128, [1, 1]), (128, [9, 4])):
        lens, d = [900, 2500], dims("bf16", H=H)
        pool, table, n_pages, rows = paged(rng, lens, 576, torch.bfloat16)
        n = sum(qs)
        q = torch.randn((n, H, 576), device=DEV).bfloat16()
        lse = torch.full((n, H), 8.0, device=DEV)
        cu, ld = i32([0, qs[0], n]), i32(lens)
        outs = [torch.zeros((2, 2500), device=DEV) for _ in range(4)]
        f = lambda out: call(d, q, lse, cu, n, max(qs), pool, n_pages, table, ld, None, 1.0, out)  # noqa: E731
        f(outs[0])
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            f(outs[1])
        torch.cuda.current_stream().wait_stream(side)
        assert torch.equal(outs[0], outs[1])
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            f(outs[2])
        ld.copy_(i32([800, 64]))
        lse.fill_(7.0)
        g.replay()
        f(outs[3])
        assert torch.equal(outs[2], outs[3]) and not torch.equal(outs[0], outs[3])
        assert status() == 0


def _bad(lens, cu, total, max_q, width, table=None, H=16):
    rng = np.random.default_rng(8)
    d = dims("bf16", H=H)
    pool, t, n, rows = paged(rng, [min(max(L, 1), 300) for L in lens], 576, torch.bfloat16, unused=0.0)
    t = t if table is None else table(t)
    q = torch.randn((total, H, 576), device=DEV).bfloat16()
    lse = torch.full((total, H), 6.0, device=DEV)
    w = torch.full((len(lens), width), 9.0, device=DEV)
    call(d, q, lse, i32(cu), total, max_q, pool, n, t, i32(lens), None, 1.0, w)
    assert status() == 5
    return d, q, lse, rows, w


@gpu
@pytest.mark.parametrize("H,bad,width", [(16, -1, 400), (16, 3, 400), (16, 100000, 400), (16, 300, 299),
                                         (128, -1, 400), (128, 3, 400), (128, 321, 400)])
def test_bad_lengths_are_left_alone(H, bad, width):
    d, q, lse, rows, w = _bad([200, bad, 90], [0, 2, 6, 9], 9, 4, width, H=H)
    assert (w[1] == 9).all()
    for b, (a, z) in ((0, (0, 2)), (2, (6, 9))):
        L = len(rows[b])
        ref, tol = reference(q[a:z], lse[a:z], rows[b], z - a, d.scale)
        assert ((w[b, :L].double() - ref).abs() <= tol + 2.0 ** -23 * ref).all()
        assert (w[b, L:] == 9).all()


@gpu
@pytest.mark.parametrize("cu,max_q", [([0, 2, 1, 5], 4), ([0, 2, 7, 99], 5), ([-3, 2, 4, 5], 4),
                                      ([0, 2, 8, 9], 5)])
def test_bad_chunks_leave_everything(cu, max_q):
    assert (_bad([200, 300, 90], cu, 9, max_q, 400)[4] == 9).all()


@gpu
def test_bad_pages_count_as_zero_rows():
    def table(t):
        t = t.clone()
        t[0, 1], t[1, 0] = -1, 1000
        return t
    d, q, lse, rows, w = _bad([200, 60], [0, 2, 4], 4, 2, 400, table)
    rows[0][64:128] = 0
    rows[1][:] = 0
    for b in range(2):
        ref, tol = reference(q[2 * b:2 * b + 2], lse[2 * b:2 * b + 2], rows[b], 2, d.scale)
        assert ((w[b, :len(ref)].double() - ref).abs() <= tol + 2.0 ** -23 * ref).all()


@gpu
def test_no_queries_at_all():
    d = dims("bf16", H=16)
    pool, table, n, _ = paged(np.random.default_rng(9), [70, 300], 576, torch.bfloat16)
    w = torch.rand((2, 300), device=DEV)
    out = torch.full((2, 300), 9.0, device=DEV)
    call(d, torch.empty((0, 16, 576), dtype=torch.bfloat16, device=DEV), torch.empty((0, 16), device=DEV),
         i32([0, 0, 0]), 0, 0, pool, n, table, i32([70, 300]), w, 0.5, out)
    assert status() == 0
    assert torch.equal(out[0, :70], 0.5 * w[0, :70]) and torch.equal(out[1], 0.5 * w[1])
    assert (out[0, 70:] == 9).all()


def test_refused_on_the_host():
    from mla_latent_kv_35_b200 import build
    build.build()
    lib = B.lib()
    x = 1 << 12

    def f(d=dims("bf16"), q=x, lse=x, cu=x, total=8, max_q=4, pool=x, n_pages=4, pt=x, mp=2, sl=x, nB=2, keep=1.0,
          wo=x, stride=128):
        return lib.mla_attn_weights(ctypes.byref(d.c()), q, lse, cu, total, max_q, pool, n_pages, pt, mp, sl, nB, 0,
                                    keep, wo, stride, 0)
    assert f(nB=0, q=0) == 0
    for kw in (dict(q=0), dict(lse=0), dict(cu=0), dict(pool=0), dict(pt=0), dict(sl=0), dict(wo=0), dict(q=x + 2),
               dict(pool=x + 8), dict(nB=-1), dict(total=-1), dict(max_q=-1), dict(max_q=9), dict(n_pages=0),
               dict(mp=0), dict(total=1 << 24), dict(mp=1 << 30), dict(mp=(1 << 25) - 1), dict(stride=0), dict(keep=float("nan")),
               dict(keep=float("inf"))):
        assert f(**kw) == 1, kw
    for d in (dims("f32"), dims("bf16", dc=256), dims("bf16", dr=32), dims("bf16", page=32)):
        assert f(d=d) == 2


@gpu
def test_binding_refuses_wrong_tensors():
    d = dims("bf16", H=4)
    pool, table, n_pages, _ = paged(np.random.default_rng(10), [70, 80], 576, torch.bfloat16)
    good = dict(q=torch.zeros((3, 4, 576), dtype=torch.bfloat16, device=DEV), lse=torch.zeros((3, 4), device=DEV),
                cu=i32([0, 1, 3]), pool=pool, table=table, lens=i32([70, 80]), wi=torch.zeros((2, 80), device=DEV),
                wo=torch.zeros((2, 80), device=DEV))

    def f(**kw):
        a = {**good, **kw}
        B.mla_attn_weights(d, a["q"], a["lse"], a["cu"], 3, 2, a["pool"], n_pages, a["table"], table.shape[1],
                           a["lens"], 2, a["wi"], 1.0, a["wo"], 80)
    f()
    for kw in (dict(q=good["q"].float()), dict(q=good["q"][:2]), dict(lse=good["lse"][:2]),
               dict(lse=good["lse"].double()), dict(cu=good["cu"][:2]), dict(pool=pool[:1]), dict(table=table[:1]),
               dict(lens=good["lens"].long()), dict(wi=good["wi"][:1]), dict(wo=good["wo"].cpu()),
               dict(wo=torch.zeros((80, 2), device=DEV).t())):
        with pytest.raises(ValueError):
            f(**kw)
    assert status() == 0
