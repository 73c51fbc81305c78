"""Tensors of more than 2^31 elements: the last rows of a call come out as they do in a
call of their own."""
import pytest
import torch

import hybrid_sliding_window_gated_b200 as swa
import sink_testutil as su

pytestmark = pytest.mark.gpu
DEV = "cuda"


@pytest.fixture(autouse=True)
def memory():
    if torch.cuda.is_available() and torch.cuda.mem_get_info()[0] < 90 << 30:
        pytest.skip("needs 90 GB of free device memory")
    yield
    torch.cuda.empty_cache()


def rand(*shape, seed=0):
    gen = torch.Generator(device=DEV).manual_seed(seed)
    return torch.empty(shape, dtype=torch.bfloat16, device=DEV).normal_(generator=gen)


def weights():
    gen = torch.Generator(device=DEV).manual_seed(9)
    return [1 + 0.1 * torch.randn(128, generator=gen, device=DEV) for _ in range(2)]


def test_forward_and_backward():
    B, T, Hq, Hkv, S = 2, 270_001, 32, 8, 4
    t = [rand(B, T, h, 128, seed=i) for i, h in enumerate((Hq, Hkv, Hkv, Hq))]
    w, dO = weights(), rand(B, T, Hq, 128, seed=5)
    assert t[0].numel() > 2 ** 31
    o, lse = swa.sink_fwd(*t, *w, S, want_lse=True)
    whole = swa.sink_bwd(*t, *w, o, lse, dO, S)
    assert swa.get_last_device_error() == (swa.OK, 0)
    last = [y[1:] for y in t]
    o1, lse1 = swa.sink_fwd(*last, *w, S, want_lse=True)
    assert torch.equal(o1[0], o[1]) and torch.equal(lse1[0], lse[1])
    part = swa.sink_bwd(*last, *w, o1, lse1, dO[1:], S)
    for a, b in zip(part[:4], whole[:4]):
        assert torch.equal(a[0], b[1])


def test_decode():
    N, Hq, Hkv, S = 17_000, 16, 8, 3
    x = [rand(N, h, 128, seed=i) for i, h in enumerate((Hq, Hkv, Hkv, Hq))]
    caches = [rand(N, Hkv, n, 128, seed=7 + i) for i, n in enumerate((128, 128, S, S))]
    assert caches[0].numel() > 2 ** 31
    pos = torch.arange(N, device=DEV) % 500
    few = [c[-3:].clone() for c in caches]
    o = swa.sink_decode_step(pos, *x, *weights(), *caches)
    o1 = swa.sink_decode_step(pos[-3:].clone(), *[y[-3:].clone() for y in x], *weights(), *few)
    assert swa.get_last_device_error() == (swa.OK, 0)
    assert torch.equal(o1, o[-3:])
    for a, b in zip(few, caches):
        assert torch.equal(a, b[-3:])


@pytest.mark.parametrize("N,P,cap", [(1, 2_200_000, 16), (60, 300, 40_000)])
def test_shared_decode(N, P, cap):
    Hq, Hkv = 16, 8
    x = [rand(N, h, 128, seed=i) for i, h in enumerate((Hq, Hkv, Hkv))]
    pre = [rand(1, Hkv, P, 128, seed=5 + i) for i in range(2)]
    own = [rand(N, Hkv, cap, 128, seed=7 + i) for i in range(2)]
    assert max(pre[0].numel(), own[0].numel()) > 2 ** 31
    pos = P + cap - 1 - torch.arange(N, device=DEV)
    o = swa.global_decode_shared(pos, *x, *weights(), *pre, P, *own, rope_base=1e4)
    joined = [torch.cat([p, c[-1:]], 2) for p, c in zip(pre, own)]
    o1 = swa.global_decode_step(pos[-1:].clone(), *[y[-1:].clone() for y in x], *weights(), *joined,
                                rope_base=1e4)
    assert swa.get_last_device_error() == (swa.OK, 0)
    # both steps' own bar is the library's 5e-3 (the shared one's 5.5e-3)
    assert su.rel(o[-1:], o1) <= 1.05e-2
