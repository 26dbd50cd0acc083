"""The operators around the cache on pages beyond 4 GB of the pool (offsets that pass 32 bits)."""

import numpy as np
import pytest
import torch

import oracle
from mla_latent_kv_35_b200 import binding as B
from gpu_util import dims, ensure_lib, status
from serving_util import DEV, bits, i32

gpu = pytest.mark.gpu
PAGES = 62000                                     # x 73728 bytes = 4.57 GB
LENS, T = [150, 70], 3


@pytest.fixture(scope="module")
def cache():
    ensure_lib()
    B.mla_get_device_status()
    d = dims("bf16", H=16)
    pool = torch.empty((PAGES, 64, 576), dtype=torch.bfloat16, device=DEV)
    table = np.array([[PAGES - 1, 58255, PAGES - 7], [PAGES - 2, 58300, 3]], np.int32)
    g = torch.Generator(device=DEV)
    g.manual_seed(0)
    for b, L in enumerate(LENS):
        for p in range(-(-L // 64)):
            pool[int(table[b, p])] = torch.randn((64, 576), generator=g, device=DEV).bfloat16()
    yield d, pool, table
    del pool
    torch.cuda.empty_cache()


def rows(pool, table, b):
    L = LENS[b]
    return torch.cat([pool[int(p)] for p in table[b, :-(-L // 64)]])[:L].double()


@gpu
def test_chunk_attention_and_weights(cache):
    d, pool, table = cache
    q = torch.randn((2 * T, 16, 576), device=DEV).bfloat16()
    cu = i32([0, T, 2 * T])
    o = torch.empty((2 * T, 16, 512), dtype=torch.bfloat16, device=DEV)
    lse = torch.empty((2 * T, 16), device=DEV)
    ws = torch.empty(B.mla_chunk_attention_workspace_size(d, 2, 2 * T, T), dtype=torch.uint8, device=DEV)
    B.mla_chunk_attention(d, q, cu, 2 * T, T, pool, PAGES, i32(table), 3, i32(LENS), 2, ws, o, lse)
    w = torch.zeros((2, 150), device=DEV)
    B.mla_attn_weights(d, q, lse, cu, 2 * T, T, pool, PAGES, i32(table), 3, i32(LENS), 2, None, 1.0, w, 150)
    assert status() == 0
    for b, L in enumerate(LENS):
        k, got = rows(pool, table, b), torch.zeros(L, dtype=torch.float64, device=DEV)
        for j in range(T):
            see = L - T + j + 1
            x = q[b * T + j].double() @ k[:see].T * d.scale
            p = torch.softmax(x, 1)
            ref, A = p @ k[:see, :512], p @ k[:see, :512].abs()
            # the stored rounding and that of P, 2^-8 each
            assert ((o[b * T + j].double() - ref).abs() <= 2.0 ** -8 * (ref.abs() + 1.1 * A)).all()
            assert (lse[b * T + j].double() - torch.logsumexp(x, 1)).abs().max() <= 2.0 ** -15
            got[:see] += (x - lse[b * T + j].double()[:, None]).exp().sum(0)
        assert ((w[b, :L].double() - got).abs() <= 2.0 ** -15 * got).all()


@gpu
def test_norm_rope_appends_there(cache):
    d, pool, table = cache
    y = torch.randn((2, 16 * 192 + 576), device=DEV).bfloat16()
    q = torch.empty((2, 16 * 192), dtype=torch.bfloat16, device=DEV)
    ckr = torch.empty((2, 576), dtype=torch.bfloat16, device=DEV)
    B.mla_norm_rope(d, y, y.shape[1], None, None, None, 1e-6, i32([9, 9]), i32([0, 1]), i32([100, 69]), i32(table),
                    3, pool, PAGES, q, 16 * 192, None, ckr, 576, 2)
    assert status() == 0
    for b, s in ((0, 100), (1, 69)):
        np.testing.assert_array_equal(bits(pool[int(table[b, s // 64]), s % 64]), bits(ckr[b]))


@gpu
def test_evict_moves_there(cache):
    d, pool, table = cache
    before = [rows(pool, table, b) for b in range(2)]
    g = torch.Generator(device=DEV)
    g.manual_seed(1)
    w = torch.rand((2, 150), generator=g, device=DEV)
    old, lens = w.cpu().numpy().copy(), i32(LENS)
    ws = torch.empty(B.mla_cache_evict_workspace_size(d, 2, 150), dtype=torch.uint8, device=DEV)
    B.mla_cache_evict(d, pool, PAGES, False, i32(table), 3, lens, 2, w, None, 150, i32([60, 33]), 2, 5, w, None, lens,
                      ws)
    assert status() == 0 and lens.tolist() == [60, 33]
    for b, new in enumerate((60, 33)):
        keep = list(range(new))
        pairs, n = oracle.evict(old[b, :LENS[b]], list(range(LENS[b])), new, 2, 5)
        assert n == new
        for to, frm in pairs:
            keep[to] = frm
        got = torch.cat([pool[int(p)] for p in table[b]])[:new].double()
        assert torch.equal(got, before[b][keep])
