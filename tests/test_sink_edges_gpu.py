"""Sink attention and the shared-prefix step where they can go wrong beyond the shapes of
test_sink_gpu.py: calls on a stream of their own, eps = 0, values near the largest bf16 and
far below their row's largest, masked values that are not finite, many CTAs and long
sequences in the backward, large norm weights, waits that run out.

Tolerances: REL and REL_DG of test_sink_gpu.py, derived there; others beside their test."""
import math

import pytest
import torch

import hybrid_sliding_window_gated_b200 as swa
import sink_testutil as su
from test_sink_gpu import REL, REL_DG, check_backward, check_forward, decode_inputs, forward, ok

pytestmark = pytest.mark.gpu
DEV = "cuda"


# ------------------------------------------------- a stream of the call's own


def wait():
    torch.cuda._sleep(int(2e8))  # about 0.1 s of the current stream


def training(seed=100):
    x = su.draw(2, 200, 4, 2, seed=seed, grad=True)
    return su.args(x, DEV), x["dO"].to(DEV)


def shared_inputs():
    N, P, cap = 40, 300, 8
    gen = torch.Generator().manual_seed(101)
    n = lambda *s: torch.randn(s, generator=gen).to(torch.bfloat16).to(DEV)
    w = [torch.ones(128, device=DEV) for _ in range(2)]
    pos = P + torch.arange(N, device=DEV) % cap
    return [pos, n(N, 4, 128), n(N, 2, 128), n(N, 2, 128), *w, n(1, 2, P, 128), n(1, 2, P, 128), P,
            n(N, 2, cap, 128), n(N, 2, cap, 128)]


def calls():
    """name -> a call that makes its own outputs and scratch on the stream it is given."""
    t, dO = training()
    o, lse = swa.sink_fwd(*t, 4, want_lse=True)
    _, wlse = swa.fwd(*t, want_lse=True)
    y, caches = decode_inputs(5, 4, 2, 4, seed=102)
    y, caches = [z.to(DEV) for z in y], [c.to(DEV) for c in caches]
    pos = torch.tensor([3, 127, 128, 200, 1000], device=DEV)
    sh = shared_inputs()
    kc = [torch.zeros(2, 2, 200, 128, dtype=torch.bfloat16, device=DEV) for _ in range(2)]
    kd = [c.expand(-1, -1, -1, -1).clone() for c in sh[9:]]
    return {
        "sink_fwd": lambda s: swa.sink_fwd(*t, 4, want_lse=True, stream=s),
        "sink_bwd": lambda s: swa.sink_bwd(*t, o, lse, dO, 4, stream=s),
        "sink_decode_step": lambda s: swa.sink_decode_step(pos, *y, *caches, stream=s),
        "global_decode_shared": lambda s: swa.global_decode_shared(*sh, rope_base=1e4, stream=s),
        "fwd": lambda s: swa.fwd(*t, want_lse=True, stream=s),
        # dwq and dwk of the window backward are sums in no fixed order
        "bwd": lambda s: swa.bwd(*t, wlse, dO, stream=s),
        "decode_step": lambda s: swa.decode_step(pos, *y, *caches[:2], stream=s),
        "global_fwd": lambda s: swa.global_fwd(*t[:3], *t[4:], *kc, want_lse=True, stream=s),
        "global_decode_step": lambda s: swa.global_decode_step(sh[0] - sh[8], *sh[1:6], *kd,
                                                               stream=s),
    }


CALLS = ["sink_fwd", "sink_bwd", "sink_decode_step", "global_decode_shared", "fwd", "bwd",
         "decode_step", "global_fwd", "global_decode_step"]


def outputs(r):
    return list(r) if isinstance(r, (tuple, list)) else [r]


def same(name, got, want):
    for i, (a, b) in enumerate(zip(got, want)):
        if name == "bwd" and i >= 4:
            torch.testing.assert_close(a, b, rtol=1e-5, atol=1e-5)
        else:
            assert torch.equal(a, b), (name, i)


@pytest.mark.parametrize("name", CALLS)
def test_stream_argument_beside_a_busy_current_stream(name):
    """What a call fills itself (dwq, dwk) is in order with the kernels that add into it."""
    call = calls()[name]
    want = [y.clone() for y in outputs(call(None))]
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    for _ in range(2):
        wait()
        got = outputs(call(s))
        s.synchronize()
        torch.cuda.synchronize()
        same(name, got, want)
    ok()


@pytest.mark.parametrize("name", CALLS)
def test_stream_argument_keeps_its_memory(name):
    """The scratch and the outputs of a call whose stream runs late go to no later
    allocation of the current stream."""
    call = calls()[name]
    want = [y.clone() for y in outputs(call(None))]
    sizes = [y.numel() * y.element_size() for y in want]
    sizes.append(swa.sink_bwd_workspace_size(2, 200, 4, 2, 4))
    sizes.append(swa.bwd_workspace_size(2, 200, 4, 2))
    sizes.append(swa.global_decode_shared_workspace_size(40, 4, 2, 300, 8))
    sizes.append(swa.global_decode_workspace_size(40, 4, 2, 8))
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(s):
        wait()
    got = outputs(call(s))
    junk = [torch.full((n,), 255, dtype=torch.uint8, device=DEV) for n in sizes for _ in range(2)]
    torch.cuda.synchronize()
    same(name, got, want)
    assert all((j == 255).all() for j in junk)
    del got, junk
    with torch.cuda.stream(s):
        wait()
    call(s)  # outputs dropped at once
    junk = [torch.full((n,), 255, dtype=torch.uint8, device=DEV) for n in sizes for _ in range(2)]
    torch.cuda.synchronize()
    assert all((j == 255).all() for j in junk)
    ok()


@pytest.mark.parametrize("name", CALLS)
def test_outputs_outlive_their_use_on_the_current_stream(name):
    call = calls()[name]
    want = [y.clone() for y in outputs(call(None))]
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    got = outputs(call(s))
    s.synchronize()
    wait()
    kept = [y.clone() for y in got]  # runs late
    sizes = [y.numel() * y.element_size() for y in got]
    del got
    with torch.cuda.stream(s):
        junk = [torch.full((n,), 255, dtype=torch.uint8, device=DEV) for n in sizes]
    torch.cuda.synchronize()
    same(name, kept, want)
    del junk
