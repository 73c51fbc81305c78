"""CPU: the 64-bit forms that the sink and shared-prefix tests compare with, pinned to
the oracle and to central differences; and what the new entry points refuse."""
import ctypes

import numpy as np
import pytest
import torch

import hybrid_sliding_window_gated_b200 as swa
import oracle
import sink_testutil as su
from hybrid_sliding_window_gated_b200 import build as swa_build


@pytest.fixture(scope="module")
def L():
    swa_build.build()
    return swa.lib()


@pytest.mark.parametrize("B,T,Hq,Hkv,R", [(1, 1, 1, 1, 42), (2, 140, 4, 2, 42), (1, 200, 3, 1, 0)])
def test_without_sinks_it_is_the_window_forward(B, T, Hq, Hkv, R):
    x = su.draw(B, T, Hq, Hkv, seed=1)
    o, lse = su.sink_forward(*su.args(x, dtype=torch.float64), 0, R, 1e4)
    f = lambda t: t.double().numpy()
    o_ref, lse_ref = oracle.fwd(f(x["q"]), f(x["k"]), f(x["v"]), f(x["g"]), f(x["wq"]), f(x["wk"]),
                                W=128, R=R, base=1e4, eps=1e-6)
    assert np.allclose(o.numpy(), o_ref, rtol=1e-9, atol=1e-11)
    assert np.allclose(lse.permute(0, 2, 1).numpy(), lse_ref, rtol=1e-9, atol=1e-11)


def test_visible_keys():
    assert su.visible(0, 4, 300) == [0]
    assert su.visible(127, 4, 300) == list(range(128))
    assert su.visible(128, 4, 300) == [0] + list(range(1, 129))  # key 0 has left the window
    assert su.visible(130, 2, 300) == [0, 1] + list(range(3, 131))
    assert su.visible(299, 16, 300) == list(range(16)) + list(range(172, 300))


def test_gradients_against_central_differences():
    B, T, Hq, Hkv, S, R = 1, 133, 2, 1, 3, 42
    x = su.draw(B, T, Hq, Hkv, seed=2, grad=True)
    t = su.args(x, dtype=torch.float64)
    grads = su.sink_gradients(t, x["dO"], S, R, 1e4)
    f = lambda y: float((su.sink_forward(*y, S, R, 1e4)[0] * x["dO"].double()).sum())
    gen = torch.Generator().manual_seed(3)
    for i, name in enumerate(su.NAMES):
        # at the sinks, in the window and past it, and a direction over all entries
        d = torch.randn(t[i].shape, generator=gen, dtype=torch.float64)
        if name in ("k", "v"):
            d[:, 4:] *= 0.1
        h = 1e-5
        up, down = list(t), list(t)
        up[i], down[i] = t[i] + h * d, t[i] - h * d
        num = (f(up) - f(down)) / (2 * h)
        ana = float((grads[i] * d).sum())
        # second-order error h^2 f''' and 64-bit cancellation eps |f| / h, both below 1e-6
        assert abs(num - ana) <= 1e-6 * max(1.0, abs(ana)), name


def _params(**kw):
    base = dict(B=1, T=256, Hq=4, Hkv=1)
    base.update(kw)
    return swa.make_params(base.pop("B"), base.pop("T"), base.pop("Hq"), base.pop("Hkv"), **base)


BAD = [
    (dict(Hq=6, Hkv=4), 4, swa.ERR_INVALID_ARG),
    (dict(rot_dim=41), 4, swa.ERR_INVALID_ARG),
    (dict(T=-1), 4, swa.ERR_INVALID_ARG),
    (dict(eps=-1.0), 4, swa.ERR_INVALID_ARG),
    (dict(), -1, swa.ERR_INVALID_ARG),
    (dict(), 17, swa.ERR_UNSUPPORTED),
    (dict(head_dim=64), 4, swa.ERR_UNSUPPORTED),
    (dict(window=64), 4, swa.ERR_UNSUPPORTED),
    (dict(rot_dim=40), 4, swa.ERR_UNSUPPORTED),
]


@pytest.mark.parametrize("kw,n_sink,code", BAD)
def test_sink_shapes_refused(L, kw, n_sink, code):
    p = _params(**kw)
    one = ctypes.c_void_p(0x1000)  # never read: the shape is refused first
    r = ctypes.byref(p)
    assert L.swa_sink_fwd(r, n_sink, *[one] * 8, None) == code
    assert L.swa_sink_bwd(r, n_sink, *[one] * 16, 1 << 40, None) == code
    assert L.swa_sink_bwd_workspace_size(r, n_sink) == 0
    if kw != dict(T=-1):  # a decode step has no T
        assert L.swa_sink_decode_step(r, n_sink, *[one] * 12, None) == code
    assert L.swa_prefill_to_sinks(r, n_sink, None, None, None, *[one] * 5, None) == code


def test_sink_pointers_refused(L):
    p = _params()
    r, ok, odd = ctypes.byref(p), 0x1000, 0x1008
    for i in range(7):  # q, k, v, g, wq, wk, o
        a = [ok] * 7
        a[i] = None
        assert L.swa_sink_fwd(r, 4, *a, None, None) == swa.ERR_INVALID_ARG
        a[i] = odd
        assert L.swa_sink_fwd(r, 4, *a, None, None) == swa.ERR_INVALID_ARG
    assert L.swa_sink_fwd(r, 4, *[ok] * 7, 0x1002, None) == swa.ERR_INVALID_ARG  # lse
    n = L.swa_sink_bwd_workspace_size(r, 4)
    assert n > 0
    for i in range(16):
        a = [ok] * 16
        a[i] = None
        assert L.swa_sink_bwd(r, 4, *a, n, None) == swa.ERR_INVALID_ARG
        a[i] = 0x1002  # below every argument's alignment
        assert L.swa_sink_bwd(r, 4, *a, n, None) == swa.ERR_INVALID_ARG
    assert L.swa_sink_bwd(r, 4, *[ok] * 16, n - 1, None) == swa.ERR_INVALID_ARG
    for i in range(12):
        a = [ok] * 12
        a[i] = None
        assert L.swa_sink_decode_step(r, 4, *a, None) == swa.ERR_INVALID_ARG
        a[i] = 0x1004
        assert L.swa_sink_decode_step(r, 4, *a, None) == swa.ERR_INVALID_ARG
    # starts and lens come together, pos0 only with them
    assert L.swa_prefill_to_sinks(r, 4, ok, None, None, *[ok] * 5, None) == swa.ERR_INVALID_ARG
    assert L.swa_prefill_to_sinks(r, 4, None, ok, None, *[ok] * 5, None) == swa.ERR_INVALID_ARG
    assert L.swa_prefill_to_sinks(r, 4, None, None, ok, *[ok] * 5, None) == swa.ERR_INVALID_ARG
    for i in range(5):
        a = [ok] * 5
        a[i] = None
        assert L.swa_prefill_to_sinks(r, 4, None, None, None, *a, None) == swa.ERR_INVALID_ARG


def test_empty_sink_calls_do_nothing(L):
    none = [None] * 8
    for kw in (dict(B=0), dict(T=0)):
        r = ctypes.byref(_params(**kw))
        assert L.swa_sink_fwd(r, 4, *none, None) == swa.OK
        assert L.swa_sink_bwd(r, 4, *[None] * 16, 0, None) == swa.OK
        assert L.swa_prefill_to_sinks(r, 4, None, None, None, *[None] * 5, None) == swa.OK
    assert L.swa_sink_decode_step(ctypes.byref(_params(B=0)), 4, *[None] * 12, None) == swa.OK
    assert L.swa_prefill_to_sinks(ctypes.byref(_params()), 0, None, None, None, *[None] * 5,
                                  None) == swa.OK


def test_decode_group_of_more_than_eight_refused(L):
    p = _params(Hq=9, Hkv=1)
    assert L.swa_sink_decode_step(ctypes.byref(p), 4, *[0x1000] * 12,
                                  None) == swa.ERR_UNSUPPORTED


def _shared(L, p, prefix_len=256, prefix_cap=256, cap=64, ptrs=None, ws=1 << 40):
    a = ptrs or [0x1000] * 12  # k_prefix, v_prefix, pos, q, k, v, wq, wk, kc, vc, o, workspace
    return L.swa_global_decode_shared(ctypes.byref(p), prefix_len, prefix_cap, *a[:10], cap, a[10],
                                      a[11], ws, None)


def test_shared_decode_refused(L):
    p = _params(window=0)
    need = L.swa_global_decode_shared_workspace_size(ctypes.byref(p), 256, 64)
    assert need > 0
    assert _shared(L, p, ws=need - 1) == swa.ERR_INVALID_ARG
    assert _shared(L, p, prefix_len=-1) == swa.ERR_INVALID_ARG
    assert _shared(L, p, prefix_cap=255) == swa.ERR_INVALID_ARG
    assert _shared(L, p, cap=0) == swa.ERR_INVALID_ARG
    assert _shared(L, p, cap=(1 << 30) + 1) == swa.ERR_UNSUPPORTED
    assert _shared(L, _params()) == swa.ERR_INVALID_ARG  # a window
    assert _shared(L, _params(window=0, Hq=9)) == swa.ERR_UNSUPPORTED
    assert _shared(L, _params(window=0, rot_dim=40)) == swa.ERR_UNSUPPORTED
    for i in range(12):
        a = [0x1000] * 12
        a[i] = None
        assert _shared(L, p, ptrs=a) == swa.ERR_INVALID_ARG
        a[i] = 0x1004
        assert _shared(L, p, ptrs=a) == swa.ERR_INVALID_ARG
    assert _shared(L, _params(window=0, B=0), ptrs=[None] * 12) == swa.OK
    size = L.swa_global_decode_shared_workspace_size
    assert size(ctypes.byref(_params()), 256, 64) == 0
    assert size(ctypes.byref(p), -1, 64) == 0 and size(ctypes.byref(p), 256, 0) == 0


def test_binding_refuses_wrong_tensors(L):
    x = su.draw(1, 8, 2, 1, seed=4)
    with pytest.raises(ValueError, match="CUDA"):
        swa.sink_fwd(*su.args(x), 4)
    with pytest.raises(TypeError, match="g is"):
        swa.sink_fwd(x["q"], x["k"], x["v"], x["g"].float(), x["wq"], x["wk"], 4)
    with pytest.raises(ValueError, match="k has"):
        swa.sink_fwd(x["q"], x["k"][:, :4], x["v"], x["g"], x["wq"], x["wk"], 4)
    z = torch.zeros(2, 1, 16, 128, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="more than one"):
        swa.global_decode_shared(torch.zeros(1, dtype=torch.int64), x["q"][:, 0], x["k"][:, 0],
                                 x["v"][:, 0], x["wq"], x["wk"], z, z, 16, z[:1], z[:1])


def test_tensors_on_another_device_refused(monkeypatch):
    monkeypatch.setattr(swa, "_current_device", lambda: 1)
    swa._on_current_device("f", torch.device("cuda", 1))
    with pytest.raises(ValueError, match="current device is cuda:1"):
        swa._on_current_device("f", torch.device("cuda", 0))
