"""mla_norm_rope against the fp64 oracle, and its refusals.

Tolerance.  One stored rounding, u |ref| (u: half a step of the type).  Before it fp32
arithmetic: a sum of n squares in at most n / 32 + 8 fp32 additions per lane and shuffle, halved
by the root: below 16 steps of 2^-24 for n <= 576; the root, its reciprocal, the products with it and
with the weight, the rotation's product and addition: below 10 more.  Together less than
26 * 2^-24 < 2^-19 of the vector's own numbers, the pair's length for a rotated number.  The
angle: reduced in fp64 and rounded to fp32, half a step of pi = 2^-23, then cos and sin within two steps:
below 2^-21 of the pair's length.
"""

import numpy as np
import pytest
import torch

import oracle
from mla_latent_kv_35_b200 import binding as B
from gpu_util import dims, ensure_lib, status
from serving_util import DEV, U, bits, i32, page_table

gpu = pytest.mark.gpu
EPS = 1e-6


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if torch.cuda.is_available():
        ensure_lib()
        B.mla_get_device_status()


def close(got, ref, dtype, pair=None):
    got, ref = got.double().cpu().numpy(), np.asarray(ref)
    size = np.abs(ref) if pair is None else pair
    err = np.abs(got - ref)
    tol = U[dtype] * np.abs(ref) + (2.0 ** -19 + 2.0 ** -21) * (1 + U[dtype]) * size + 1e-38
    assert (err <= tol).all(), (err.max(), (err / np.maximum(tol, 1e-300)).max())


def pairs_of(x):
    p = np.sqrt(x[..., 0::2] ** 2 + x[..., 1::2] ** 2)
    return np.repeat(p, 2, -1)


def run(d, T, seed=0, pad=0, q_pad=0, weights="qck", use_qbuf=True, use_pool=True, use_ckr=False,
        inplace=False, shift=0, scale=1.0):
    rng = np.random.default_rng(seed)
    dt = d.torch_dtype
    H, dn, dr, dc = d.n_heads, d.d_nope, d.d_rope, d.d_latent
    dqk, D = dn + dr, dc + dr
    Y = H * dqk + D + pad
    store = torch.full((T * Y + shift,), float("nan"), dtype=dt, device=DEV)
    y = store[shift:].view(T, Y)
    x = torch.from_numpy((scale * rng.standard_normal((T, H * dqk + D))).astype(np.float32)).to(dt)
    y[:, :H * dqk + D] = x.to(DEV)
    before = y.clone()
    mk = lambda n: torch.from_numpy((1 + .3 * rng.standard_normal(n)).astype(np.float32)).to(dt)  # noqa: E731
    w_q, w_c, w_kr = (mk(n) if f in weights else None for n, f in ((dqk, "q"), (dc, "c"), (dr, "k")))
    nseq, per = max(1, T // 5), 2 * d.page_size + 3
    table, n_pages = page_table(rng, [per] * nseq, d.page_size)
    place = rng.choice(nseq * per, T, replace=False)
    batch, slot = place // per, place % per
    pos = rng.integers(0, 131072, T)
    pos[0] = 131071
    pool = torch.full((n_pages, d.page_size, D), 7.0, dtype=dt, device=DEV) if use_pool else None
    qs = Y if inplace else H * dqk + q_pad
    q = y if inplace else torch.full((T, qs), 5.0, dtype=dt, device=DEV)
    qbuf = torch.full((T, H, D), 3.0, dtype=dt, device=DEV) if use_qbuf else None
    ckr = (y[:, H * dqk:] if inplace else torch.full((T, D + pad), 2.0, dtype=dt, device=DEV)) if use_ckr else None
    dev = lambda w: None if w is None else w.to(DEV)  # noqa: E731
    B.mla_norm_rope(d, y, Y, dev(w_q), dev(w_c), dev(w_kr), EPS, i32(pos), i32(batch), i32(slot),
                    i32(table), table.shape[1], pool, n_pages, q, qs, qbuf, ckr,
                    (Y if inplace else D + pad) if use_ckr else 0, T)
    assert status() == 0
    f = lambda w: None if w is None else w.double().numpy()  # noqa: E731
    rq, rk = oracle.norm_rope(x.double().numpy(), H, dn, dr, dc, f(w_q), f(w_c), f(w_kr), EPS, pos)
    gq = q[:, :H * dqk].reshape(T, H, dqk)
    close(gq[..., :dn], rq[..., :dn], dt)
    if use_qbuf:
        close(qbuf[..., dc:], rq[..., dn:], dt, pairs_of(rq[..., dn:]))
        assert (qbuf[..., :dc] == 3).all()                       # mla_absorb_q's part
        if not inplace:
            assert (gq[..., dn:] == 5).all()
    else:
        close(gq[..., dn:], rq[..., dn:], dt, pairs_of(rq[..., dn:]))
    if q_pad and not inplace:
        assert (q[:, H * dqk:] == 5).all()
    if inplace:                                                   # nothing else of y changes
        a, b = bits(y), bits(before)
        np.testing.assert_array_equal(a[:, H * dqk + D:], b[:, H * dqk + D:])
        if not use_ckr:
            np.testing.assert_array_equal(a[:, H * dqk:], b[:, H * dqk:])
    else:
        np.testing.assert_array_equal(bits(y), bits(before))
    got = []
    if use_pool:
        page = torch.from_numpy(table[batch, slot // d.page_size]).long().to(DEV)
        sl = torch.from_numpy(slot % d.page_size).to(DEV)
        got.append(pool[page, sl].clone())
        pool[page, sl] = 7.0
        assert (pool == 7).all()                                  # no other slot was written
    if use_ckr:
        got.append(ckr[:, :D])
        if not inplace and pad:
            assert (ckr[:, D:] == 2).all()
    for g in got:
        close(g[:, :dc], rk[:, :dc], dt)
        if dr:
            close(g[:, dc:], rk[:, dc:], dt, pairs_of(rk[:, dc:]))
    if len(got) == 2:
        np.testing.assert_array_equal(bits(got[0]), bits(got[1]))
    return q, pool


WIDE = [(dt, H) for dt in ("bf16", "f32") for H in (1, 5, 32, 33, 128)]


@gpu
@pytest.mark.parametrize("dtype,H", WIDE)
@pytest.mark.parametrize("T", [1, 9])
def test_deepseek_widths(dtype, H, T):
    run(dims(dtype, H=H), T, seed=H + T)
    run(dims(dtype, H=H), T, seed=H + T, use_qbuf=False, pad=16, q_pad=8)


@gpu
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_many_tokens(dtype):
    run(dims(dtype, H=16), 1031, seed=5)


@gpu
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("weights", ["", "q", "c", "k", "qc"])
def test_parts_without_norm(dtype, weights):
    run(dims(dtype, H=6), 7, seed=3, weights=weights, use_ckr=True)


@gpu
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("use_qbuf", [True, False])
@pytest.mark.parametrize("use_ckr", [True, False])
def test_in_place(dtype, use_qbuf, use_ckr):
    run(dims(dtype, H=12), 21, seed=4, inplace=True, use_qbuf=use_qbuf, use_ckr=use_ckr, pad=24)
    # the kernel for any layout
    run(dims(dtype, H=3), 5, seed=4, inplace=True, use_qbuf=use_qbuf, use_ckr=use_ckr, pad=1)


@gpu
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("dn,dr,dc,page", [(32, 16, 64, 64), (3, 2, 5, 16), (40, 0, 33, 7),
                                           (128, 64, 512, 16), (96, 96, 256, 64)])
def test_other_widths(dtype, dn, dr, dc, page):
    d = dims(dtype, H=3, dn=dn, dc=dc, dr=dr, dm=64, page=page)
    run(d, 11, seed=6, use_ckr=True, weights="qck" if dr else "qc")
    run(d, 1, seed=7, use_pool=False, use_ckr=True, use_qbuf=False, pad=1, weights="qck" if dr else "qc")


@gpu
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_unaligned_rows_take_the_other_kernel_and_agree(dtype):
    d = dims(dtype, H=7)
    run(d, 6, seed=8, pad=3, q_pad=1)
    run(d, 6, seed=8, shift=1)


@gpu
def test_large_and_tiny_numbers():
    run(dims("f32", H=4), 3, seed=9, scale=1e15)
    run(dims("f32", H=4), 3, seed=9, scale=1e-15)
    run(dims("bf16", H=4), 3, seed=9, scale=1e-4)


@gpu
def test_two_kernels_agree_on_no_pool_and_zero_rows():
    d = dims("bf16", H=4)
    y = torch.zeros((2, 4 * 192 + 576), dtype=torch.bfloat16, device=DEV)
    w = torch.ones(512, dtype=torch.bfloat16, device=DEV)
    q = torch.full((2, 4 * 192), 9.0, dtype=torch.bfloat16, device=DEV)
    ckr = torch.full((2, 576), 9.0, dtype=torch.bfloat16, device=DEV)
    B.mla_norm_rope(d, y, y.shape[1], w[:192], w, w[:64], EPS, i32([0, 5]), None, None, None, 0,
                    None, 0, q, 768, None, ckr, 576, 2)
    assert status() == 0
    assert (q == 0).all() and (ckr == 0).all()
    B.mla_norm_rope(d, y, y.shape[1], None, None, None, EPS, i32([0, 5])[:0], None, None, None, 0,
                    None, 0, q, 768, None, None, 0, 0)           # no tokens


@gpu
@pytest.mark.parametrize("field,value", [("batch", -1), ("batch", 2), ("slot", -1), ("slot", 128),
                                         ("page", -1), ("page", 9)])
@pytest.mark.parametrize("H", [4, 3])
def test_bad_places_are_skipped_and_reported(field, value, H):
    d = dims("bf16", H=H)
    pad = 0 if H == 4 else 1                                      # both kernels
    Y = H * 192 + 576 + pad
    y = torch.randn((3, Y), device=DEV).bfloat16()
    batch, slot, table = [0, 1, 0], [5, 70, 64], np.array([[0, 1], [2, 3]])
    if field == "batch":
        batch[1] = value
    elif field == "slot":
        slot[1] = value
    else:
        table[1, 1] = value
    pool = torch.full((4, 64, 576), 7.0, dtype=torch.bfloat16, device=DEV)
    q = torch.empty((3, H * 192), dtype=torch.bfloat16, device=DEV)
    B.mla_norm_rope(d, y, Y, None, None, None, EPS, i32([1, 2, 3]), i32(batch), i32(slot),
                    i32(table), 2, pool, 4, q, H * 192, None, None, 0, 3)
    assert status() == 5
    pool[0, 5] = 7.0
    pool[1, 0] = 7.0
    assert (pool == 7).all()


@gpu
def test_graph_replay_and_other_stream():
    d = dims("bf16", H=8)
    T, Y = 4, 8 * 192 + 576
    y = torch.randn((T, Y), device=DEV).bfloat16()
    w = torch.ones(192, dtype=torch.bfloat16, device=DEV)
    q = torch.zeros((T, 8 * 192), dtype=torch.bfloat16, device=DEV)
    ckr = torch.zeros((T, 576), dtype=torch.bfloat16, device=DEV)
    pos = i32([1, 2, 3, 4])
    call = lambda out: B.mla_norm_rope(d, y, Y, w, None, None, EPS, pos, None, None, None, 0, None,  # noqa: E731
                                       0, out, 8 * 192, None, ckr, 576, T)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        call(q)
    torch.cuda.current_stream().wait_stream(side)
    g = torch.cuda.CUDAGraph()
    q2 = torch.zeros_like(q)
    with torch.cuda.graph(g):
        call(q2)
    want = torch.zeros_like(q)
    g.replay()
    call(want)
    assert torch.equal(q2, q) and torch.equal(q2, want)            # any stream, the same bits
    y.mul_(1.5)                                                    # a replay reads what y holds
    g.replay()
    call(want)
    assert torch.equal(want, q2) and not torch.equal(q2, q)


def test_refused_on_the_host():
    lib = ensure_lib_cpu()
    import ctypes
    ok = dims("bf16", H=2)

    def call(d=ok, y=1 << 12, ys=960, eps=1e-6, pos=1 << 12, n_seqs=1, mp=1, pool=0, n_pages=1,
             q=1 << 12, qs=384, ckr=0, cs=576, T=3, slot=0):
        return lib.mla_norm_rope(ctypes.byref(d.c()), y, ys, 0, 0, 0, eps, pos, slot, slot, slot,
                                 n_seqs, mp, pool, n_pages, q, qs, 0, ckr, cs, T, 0)
    assert call(T=0, y=0, q=0, pos=0) == 0
    for kw in (dict(T=-1), dict(eps=0.0), dict(eps=-1.0), dict(eps=float("nan")),
               dict(eps=float("inf")), dict(ys=959), dict(qs=383), dict(ckr=1 << 12, cs=575),
               dict(y=0), dict(q=0), dict(pos=0), dict(pool=1 << 12), dict(pool=1 << 12, mp=0),
               dict(pool=1 << 12, slot=1 << 12, n_pages=0),
               dict(pool=1 << 12, slot=1 << 12, n_seqs=0), dict(d=dims("bf16", H=0))):
        assert call(**kw) == 1, kw


def ensure_lib_cpu():
    from mla_latent_kv_35_b200 import build
    build.build()
    return B.lib()


@gpu
def test_binding_refuses_wrong_tensors():
    d = dims("bf16", H=2)
    Y = 2 * 192 + 576
    good = dict(y=torch.zeros((3, Y), dtype=torch.bfloat16, device=DEV), ys=Y,
                w=torch.ones(192, dtype=torch.bfloat16, device=DEV), pos=i32([1, 2, 3]),
                q=torch.zeros((3, 384), dtype=torch.bfloat16, device=DEV), qbuf=None)

    def call(**kw):
        a = {**good, **kw}
        B.mla_norm_rope(d, a["y"], a["ys"], a["w"], None, None, EPS, a["pos"], None, None, None, 0,
                        None, 0, a["q"], 384, a["qbuf"], None, 0, 3)
    call()
    for kw in (dict(y=good["y"].cpu()), dict(y=good["y"].float()), dict(y=good["y"][:2].clone()),
               dict(w=good["w"][:191]), dict(w=good["w"].float()), dict(pos=good["pos"][:2]),
               dict(pos=good["pos"].long()), dict(q=good["q"][:2].clone()),
               dict(qbuf=torch.zeros((3, 2, 575), dtype=torch.bfloat16, device=DEV)),
               dict(pos=torch.zeros(6, dtype=torch.int32, device=DEV)[::2])):
        with pytest.raises(ValueError):
            call(**kw)
    assert status() == 0
