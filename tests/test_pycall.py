"""CPU checks of the native Python calls: what they accept, refuse and pass on.

The calls take the current device from binding._where; here it is replaced by that of CPU tensors, and
every call that reaches the library has no work to do (no tokens or no sequences), so that nothing is
launched."""

import pytest
import torch

from mla_latent_kv_35_b200 import binding as B

H, DN, DC, DR, DV, DM, PAGE = 4, 16, 32, 8, 16, 64, 64
DQK, D = DN + DR, DC + DR


def dims(dtype="bf16"):
    return B.MLADims(H, DN, DC, DR, DV, DM, PAGE, 0.1, 10000.0, dtype)


@pytest.fixture(autouse=True)
def _cpu(monkeypatch):
    from mla_latent_kv_35_b200 import build
    build.build()
    B.lib()
    monkeypatch.setattr(B, "_where", lambda: (-1, 0))


def z(*s, dt=torch.bfloat16):
    return torch.zeros(s, dtype=dt)


def i32(*s):
    return torch.zeros(s, dtype=torch.int32)


def f32(*s):
    return torch.zeros(s)


def u8(n):
    return torch.zeros(n, dtype=torch.uint8)


# name -> (arguments after dims, the places of its tensors with a size of their own)
def norm_args(T=0):
    Y = H * DQK + D
    return [z(3, Y), Y, z(DQK), z(DC), z(DR), 1e-6, i32(3), i32(3), i32(3), i32(2, 5), 5, z(4, PAGE, D), 4,
            z(3, H * DQK), H * DQK, z(3, H, D), z(3, D), D, T]


def chunk_args(total=0):
    return [z(3, H, D), i32(3), total, 0, z(4, PAGE, D), 4, i32(2, 5), 5, i32(2), 2, u8(64), z(3, H, DC),
            f32(3, H)]


def weights_args(nB=0):
    return [z(3, H, D), f32(3, H), i32(3), 0, 0, z(4, PAGE, D), 4, i32(2, 5), 5, i32(2), nB, f32(2, 9), 1.0,
            f32(2, 9), 9]


def out_args(T=0):
    return [z(3, H, DC), z(H, DV, DC), z(DM, H * DV), u8(1 << 16), f32(3, DM), T]


def evict_args(nB=0):
    return [z(4, PAGE, D), 4, False, i32(2, 5), 5, i32(2), nB, f32(2, 9), i32(2, 9), 9, i32(2), 0, 0, f32(2, 9),
            i32(2, 9), i32(2), u8(1 << 16)]


CALLS = {"norm": (B.mla_norm_rope, norm_args), "out": (B.mla_out_proj_bf16, out_args),
         "evict": (B.mla_cache_evict, evict_args), "weights": (B.mla_attn_weights, weights_args),
         "chunk": (B.mla_chunk_attention, chunk_args)}


def call(name, args, dtype="bf16"):
    f, _ = CALLS[name]
    f(dims(dtype), *args)


@pytest.mark.parametrize("name", ["norm", "out", "evict"])
def test_calls_without_work_return(name):
    call(name, CALLS[name][1]())


@pytest.mark.parametrize("name", ["weights", "chunk"])
def test_the_librarys_refusal_comes_back(name):
    with pytest.raises(B.MLAError) as e:               # these widths have no tensor-core kernel
        call(name, CALLS[name][1]())
    assert e.value.code == 2


@pytest.mark.parametrize("name", list(CALLS))
def test_every_tensor_is_checked(name):
    good = CALLS[name][1]()
    for k, x in enumerate(good):
        if not isinstance(x, torch.Tensor):
            continue
        wrong = [x.double(), torch.empty(x.shape, dtype=x.dtype, device="meta")]
        if x.dim() > 1 and not (name == "norm" and k in (0, 13, 16)):       # not the rows at a stride
            wrong.append(x.transpose(0, 1))
        for bad in wrong:
            with pytest.raises(ValueError):
                call(name, good[:k] + [bad] + good[k + 1:])
        for bad in (None, 5):
            if bad is None and (name, k) in {("norm", 2), ("norm", 3), ("norm", 4), ("norm", 11), ("norm", 15),
                                             ("norm", 16), ("weights", 11), ("evict", 8), ("evict", 14)}:
                continue                               # may be left out
            with pytest.raises(TypeError):
                call(name, good[:k] + [bad] + good[k + 1:])


@pytest.mark.parametrize("name", list(CALLS))
def test_tensors_of_another_device(name, monkeypatch):
    monkeypatch.setattr(B, "_where", lambda: (0, 0))
    with pytest.raises(ValueError, match="must live on the current CUDA device"):
        call(name, CALLS[name][1]())


@pytest.mark.parametrize("name,k,cut", [
    ("norm", 2, 1), ("norm", 3, 1), ("norm", 4, 1), ("norm", 11, 1), ("out", 1, 1), ("out", 2, 1),
    ("evict", 0, 1), ("weights", 5, 1), ("chunk", 4, 1)])
def test_too_small_whatever_the_number_of_tokens(name, k, cut):
    good = CALLS[name][1]()
    with pytest.raises(ValueError):
        call(name, good[:k] + [good[k][:-cut]] + good[k + 1:])


@pytest.mark.parametrize("name,n,ks", [
    ("norm", 4, (0, 6, 7, 8, 13, 15, 16)), ("out", 4, (0, 4)), ("evict", 3, (3, 5, 7, 8, 10, 13, 14, 15)),
    ("weights", 3, (2, 7, 9, 11, 13)), ("chunk", 4, (0, 11, 12))])
def test_too_small_for_the_tokens_or_sequences(name, n, ks):
    """One more than the tensors hold: each one is found, the ones before it being large enough."""
    f, make = CALLS[name]
    big = make(n)
    for k, x in enumerate(big):
        if isinstance(x, torch.Tensor):
            big[k] = torch.zeros((2 * x.numel(),), dtype=x.dtype) if name != "norm" or k not in (0, 13, 16) else \
                torch.zeros((2 * x.shape[0], x.shape[1]), dtype=x.dtype)
    for k in ks:
        args = list(big)
        args[k] = make(n)[k]
        with pytest.raises(ValueError):
            call(name, args)


def test_rows_of_a_wider_tensor():
    """q, y and ckr are rows at a stride, held by the storage behind a view."""
    Y = H * DQK + D
    a = norm_args()
    y = z(3, Y + 7)
    a[0], a[1] = y[:, 3:], Y + 7
    call("norm", a)                                    # no rows: whatever the view holds
    a[-1] = 3
    for k in (6, 7, 8):
        a[k] = i32(3)
    with pytest.raises(ValueError, match="y: the tensor does not hold 3 rows"):
        call("norm", [z(3, Y - 1)] + a[1:])
    with pytest.raises(ValueError, match="y: the tensor does not hold 3 rows"):
        call("norm", [y[:, 8:]] + a[1:])               # one number past the storage's end
    a[16], a[17] = z(3, D)[:, 1:], D
    with pytest.raises(ValueError, match="ckr: the tensor does not hold 3 rows"):
        call("norm", a)


def test_integers_must_fit_and_be_integers():
    a = out_args()
    with pytest.raises(ValueError):
        call("out", a[:-1] + [1 << 31])
    with pytest.raises(TypeError):
        call("out", a[:-1] + [1.5])
    with pytest.raises(OverflowError):
        call("out", a[:-1] + [1 << 70])
    with pytest.raises(TypeError):
        B._native().out_proj_bf16(1, 2)
    with pytest.raises(B.MLAError):
        call("out", a[:-1] + [-1])


def test_dtype_follows_the_dims():
    a = norm_args()
    with pytest.raises(ValueError, match="expected Float, got BFloat16"):
        call("norm", a, "f32")
    call("norm", [x.float() if isinstance(x, torch.Tensor) and x.dtype == torch.bfloat16 else x for x in a], "f32")


def test_a_tensor_without_memory_raises():
    """A C++ exception (a sparse tensor has no storage) arrives as a Python one."""
    a = out_args()
    with pytest.raises((RuntimeError, ValueError)):
        call("out", [a[0].to_sparse()] + a[1:])
    b = norm_args()
    with pytest.raises((RuntimeError, ValueError)):
        call("norm", [b[0].to_sparse()] + b[1:])


def test_failed_calls_leak_no_references():
    import sys
    a = norm_args()
    before = [sys.getrefcount(x) for x in a]
    for _ in range(50):
        call("norm", a)
        for k in range(len(a)):
            if isinstance(a[k], torch.Tensor):
                with pytest.raises(ValueError):
                    call("norm", a[:k] + [a[k].double()] + a[k + 1:])
    assert [sys.getrefcount(x) for x in a] == before
