"""CPU checks of the binding: what its calls hand to the library, and what it needs to load."""

import ctypes
import sys
import threading

import pytest
import torch

from mla_latent_kv_35_b200 import binding as B


def dims(cls=B.MLADims):
    return cls(4, 16, 32, 8, 16, 64, 64, 0.1, 10000.0, "bf16")


def n_heads_at(addr):
    return ctypes.cast(addr, ctypes.POINTER(B.Dims)).contents.n_heads


def test_two_first_calls_at_once_share_one_struct():
    """A second first call that comes in between finding no struct and keeping one: both calls hold the
    struct that is kept."""
    inner = []

    class Slow(B.MLADims):
        def c(self):
            if not inner:
                inner.append(None)
                inner[0] = B._addr(self)               # the other thread's whole call
            return super().c()
    d = dims(Slow)
    outer = B._addr(d)
    assert outer == inner[0] == B._addr(d)
    assert n_heads_at(outer) == 4


def test_first_calls_of_four_threads():
    old = sys.getswitchinterval()
    sys.setswitchinterval(1e-6)
    try:
        for _ in range(300):
            d, seen, go = dims(), [], threading.Barrier(4)

            def first():
                go.wait()
                seen.append(B._addr(d))
            ts = [threading.Thread(target=first) for _ in range(4)]
            for t in ts:
                t.start()
            for t in ts:
                t.join()
            assert len(seen) == 4 and set(seen) == {B._addr(d)}
    finally:
        sys.setswitchinterval(old)


H, DN, DC, DR, PAGE = 4, 16, 32, 8, 64
DQK, D = DN + DR, DC + DR
Y = H * DQK + D


@pytest.fixture
def norm(monkeypatch):
    """norm(T=, y=, ...) calls mla_norm_rope on CPU tensors.  It reaches the library only with an eps that
    the library refuses, so nothing is launched."""
    from mla_latent_kv_35_b200 import build
    build.build()
    monkeypatch.setattr(B, "_where", lambda: (-1, 0))

    def call(T=3, **kw):
        z = lambda *s: torch.zeros(s, dtype=torch.bfloat16)  # noqa: E731
        a = dict(y=z(T, Y), ys=Y, q=z(T, H * DQK), qs=H * DQK, ckr=None, cs=0)
        a.update(kw)
        B.mla_norm_rope(dims(), a["y"], a["ys"], None, None, None, -1.0, torch.zeros(T, dtype=torch.int32), None,
                        None, None, 0, None, 0, a["q"], a["qs"], None, a["ckr"], a["cs"], T)
    return call


def rows(n, width, wide=0):
    return torch.zeros((n, width + wide), dtype=torch.bfloat16)[:, :width]


@pytest.mark.parametrize("name,stride,width", [("y", "ys", Y), ("q", "qs", H * DQK), ("ckr", "cs", D)])
def test_rows_at_a_stride_lie_within_their_tensor(norm, name, stride, width):
    def refused(t, s, T=3):
        with pytest.raises(ValueError, match=f"{name}: the tensor does not hold {T} rows"):
            norm(T, **{name: t, stride: s})

    def reaches_the_library(t, s, T=3):
        with pytest.raises(B.MLAError):
            norm(T, **{name: t, stride: s})
    big = rows(8, width + 5)
    reaches_the_library(rows(3, width), width)
    reaches_the_library(rows(3, width, 9), width + 9)                    # a view of wider rows
    reaches_the_library(big[:, 5:], width + 5, 8)                        # which end with the storage
    reaches_the_library(big[2:5, 5:], width + 5)
    reaches_the_library(big.view(-1)[:2 * (width + 5) + width], width + 5)   # flat, the last row short
    reaches_the_library(rows(3, width).view(3, -1, 1, width // 2), width)
    reaches_the_library(big[1:2, 5:], width, 1)                          # one row: any stride
    reaches_the_library(big[1:3, 5:], width, 1)
    reaches_the_library(big.view(2, 4, -1)[..., 5:], width + 5, 8)       # tokens in two dimensions
    reaches_the_library(big.view(2, 4, -1)[..., 5:].view(2, 4, 2, -1), width + 5, 8)
    reaches_the_library(big.view(8, 1, -1)[..., 5:], width + 5, 8)
    refused(big.view(2, 4, -1)[:, :3, 5:], width + 5, 6)                 # not at one stride
    refused(big.view(2, 4, -1)[..., 5:], width + 5, 9)
    refused(big.view(2, 4, -1).transpose(0, 1)[..., 5:], width + 5, 8)
    refused(big[:2], width + 5)                                          # fewer rows than tokens
    refused(big[:2, 5:], width + 5)
    refused(big.view(-1)[:2 * (width + 5) + width - 1], width + 5)
    refused(big[:, 6:], width + 5)                                       # rows too short
    refused(big[:, 5:], width)                                           # not the view's stride
    refused(big[::2, 5:], width + 5)
    refused(rows(width, 3).t(), width)                                   # columns as rows
    refused(rows(3, 2 * width)[:, ::2], 2 * width)                       # every other number
    refused(rows(1, width).expand(3, width), width)                      # one row for all
    reaches_the_library(big[:0], width, 0)


@pytest.mark.parametrize("fp8", [0, 1])
def test_eviction_refuses_a_pool_at_an_odd_address(fp8):
    """A slice of a uint8 tensor may begin at any byte; rows move in units of two bytes at least."""
    from mla_latent_kv_35_b200 import build
    build.build()
    d = B.MLADims(4, 128, 512, 64, 128, 64, 64, 0.1, 10000.0, "bf16")
    x = 1 << 12
    for pool in (x + 1, x + 15):
        assert B.lib().mla_cache_evict(ctypes.byref(d.c()), pool, 4, fp8, x, 2, x, 2, x, 0, 100, x, 0, 0, x, 0, x,
                                       x, 1 << 20, 0) == 1


def test_tensor_core_softmaxes_refuse_a_negative_scale():
    """They scale a block's greatest product, which is its least score then; the decode has another
    kernel for it, and the gathered weights take no maximum."""
    from mla_latent_kv_35_b200 import build
    build.build()
    lib, x = B.lib(), 1 << 12
    for scale, refused in ((-0.1, True), (0.0, False), (0.1, False)):
        d = B.MLADims(16, 128, 512, 64, 128, 64, 64, scale, 10000.0, "bf16")
        c = ctypes.byref(d.c())
        # zero sequences, or a workspace that is too small: nothing is launched
        want = 2 if refused else 0
        assert lib.mla_chunk_attention(c, 0, 0, 0, 0, 0, 4, 0, 2, 0, 0, 0, 0, 0, 0, 0) == want
        assert lib.mla_decode_fp8(c, 0, 0, 4, 0, 2, 0, 0, 1, 0, 0, 0, 0, 0, 0) == want
        assert lib.mla_prefill_attention(c, 0, 16 * 192, 0, 0, 0, 0, 8, 0, 0, 0) == want
        assert lib.mla_attn_weights(c, 0, 0, 0, 0, 0, 0, 4, 0, 2, 0, 0, 0, 1.0, 0, 128, 0) == 0
        assert (B.mla_chunk_attention_workspace_size(d, 2, 8, 4) == 0) == refused
        assert (B.mla_decode_fp8_workspace_size(d, 2, 1) == 0) == refused
        assert B.mla_decode_config(d, 1)[0] == (B.DECODE_KERNEL_SIMT if refused else B.DECODE_KERNEL_TC)
    assert lib.mla_chunk_attention(ctypes.byref(B.MLADims(16, 128, 512, 64, 128, 64, 64, -0.1, 1e4, "bf16").c()),
                                   x, x, 8, 4, x, 4, x, 2, x, 2, x, 1 << 40, x, x, 0) == 2


def test_the_library_loads_without_the_native_calls(monkeypatch):
    """Only the calls that go through the extension need it; they say what is missing."""
    from mla_latent_kv_35_b200 import build
    build.build()
    monkeypatch.setitem(sys.modules, "mla_latent_kv_35_b200._pycall", None)      # its import fails
    import mla_latent_kv_35_b200 as pkg
    monkeypatch.delattr(pkg, "_pycall", raising=False)
    monkeypatch.setattr(B, "_lib", None)
    monkeypatch.setattr(B, "_pycall", None)
    assert B.mla_status_string(0) == "ok"
    assert B.mla_decode_workspace_size(dims(), 2, 1) > 0
    assert B.mla_cache_evict_workspace_size(dims(), 2, 100) > 0
    monkeypatch.setattr(B, "_where", lambda: (-1, 0))
    with pytest.raises(ImportError, match="mla_latent_kv_35_b200.build"):
        B.mla_out_proj_bf16(dims(), None, None, None, None, None, 0)


def test_native_calls_of_another_python_or_torch_are_built_again(monkeypatch, tmp_path):
    import shutil
    from mla_latent_kv_35_b200 import build
    build.build()
    assert build.calls_up_to_date()
    lib = {t: (tmp_path / n) for t, n in (("CALLS", "_pycall.so"), ("CALLS_STAMP", "stamp"))}
    for t, p in lib.items():
        shutil.copy2(getattr(build, t), p)
        monkeypatch.setattr(build, t, str(p))
    built = []
    monkeypatch.setattr(build, "_compile", lambda cmd, target, verbose: built.append(target))
    build.build()
    assert built == []
    for name in ("torch", "python"):
        with monkeypatch.context() as m:
            if name == "torch":
                m.setattr(torch, "__version__", "0.0.0")
            else:
                m.setattr(sys, "version", "0.0.0")
            assert not build.calls_up_to_date()
            built.clear()
            build.build()
            assert built == [build.CALLS] and build.calls_up_to_date()
        assert not build.calls_up_to_date()            # the stamp is the other one's now
        build.build()
    lib["CALLS_STAMP"].unlink()
    assert not build.calls_up_to_date()


@pytest.mark.parametrize("H,dm,most", [(1, 64, 1100), (16, 5120, 1100), (128, 5120, 140)])
def test_memory_of_the_buffers_of_many_step_lengths(H, dm, most):
    """Steps of every length up to `most` hold at most five times what the longest one needs by itself."""
    import numpy as np
    from mla_latent_kv_35_b200 import build
    from mla_latent_kv_35_b200.engine import MLADecodeLayer
    build.build()
    d = B.MLADims(H, 128, 512, 64, 128, dm, 64, 0.1, 10000.0, "bf16")
    none = np.zeros((0, 1), np.float32)
    layer = MLADecodeLayer(d, {k: none for k in ("W_Q", "W_DKV", "W_KR", "W_UK", "W_UV", "W_O")}, "cpu")

    def held():
        s = {}
        for v in layer._bufs.values():
            for t in v.values() if isinstance(v, dict) else [v]:
                s[t.untyped_storage().data_ptr()] = t.untyped_storage().nbytes()
        return sum(s.values())
    for nB in (1, 64):
        T = 1
        while T <= most:
            bf = layer.extend_buffers(nB, T, T)
            assert bf["ws"].numel() >= B.mla_chunk_attention_workspace_size(d, nB, T, T)
            assert bf["scratch"].numel() >= B.mla_out_proj_bf16_scratch_size(d, T)
            row = 2 * (layer.Y + H * (576 + 512)) + 4 * (H + dm)
            alone = (T * row + B.mla_chunk_attention_workspace_size(d, nB, T, T) +
                     B.mla_out_proj_bf16_scratch_size(d, T))
            assert held() <= 5 * alone, (nB, T, held() / alone)
            T += max(1, T // 5)
        layer._bufs.clear()
