"""GPU parity of the shared-prefix decode step with a plain 64-bit form.

Tolerance: o is bf16 (2^-8 of a value at most), P of the prefix part is bf16 as well
(2^-8 of a term; random signs make it no more than that of the sum in the 2-norm), q'
carries 16 bits: sqrt(2) 2^-8 = 5.5e-3 bounds the relative 2-norm."""
import pytest
import torch

import hybrid_sliding_window_gated_b200 as swa
import sink_testutil as su

pytestmark = pytest.mark.gpu
DEV = "cuda"
REL = 5.5e-3


def inputs(N, Hq, Hkv, P, pcap, cap, seed, kstd=1.0):
    gen = torch.Generator().manual_seed(seed)
    n = lambda *s, std=1.0: (torch.randn(s, generator=gen) * std).to(torch.bfloat16)
    return dict(q=n(N, Hq, 128), k=n(N, Hkv, 128), v=n(N, Hkv, 128),
                wq=1 + 0.1 * torch.randn(128, generator=gen),
                wk=1 + 0.1 * torch.randn(128, generator=gen),
                kp=n(1, Hkv, pcap, 128, std=kstd), vp=n(1, Hkv, pcap, 128),
                kc=n(N, Hkv, cap, 128, std=kstd), vc=n(N, Hkv, cap, 128))


def reference(x, pos, P, R, base):
    q = su.norm_rope(x["q"].double(), x["wq"].double(), pos, R, base)
    k = su.norm_rope(x["k"].double(), x["wk"].double(), pos, R, base).to(torch.bfloat16)
    out = torch.empty(q.shape, dtype=torch.float64)
    for n, p in enumerate(pos.tolist()):
        x["kc"][n, :, p - P], x["vc"][n, :, p - P] = k[n], x["v"][n]
        cat = lambda a, b: torch.cat([a[0, :, :P], b[n, :, :p - P + 1]], 1).double()
        out[n] = su.context_attention(q[n], cat(x["kp"], x["kc"]), cat(x["vp"], x["vc"]))
    return out


def step(x, pos, P, R=42, base=1e4, **kw):
    d = {n: t.to(DEV) for n, t in x.items()}
    o = swa.global_decode_shared(pos.to(DEV), d["q"], d["k"], d["v"], d["wq"], d["wk"], d["kp"],
                                 d["vp"], P, d["kc"], d["vc"], rot_dim=R, rope_base=base, **kw)
    return o, d


def check(N, Hq, Hkv, P, pcap, cap, R=42, seed=0, kstd=1.0):
    x = inputs(N, Hq, Hkv, P, pcap, cap, seed, kstd)
    gen = torch.Generator().manual_seed(seed + 1)
    pos = P + torch.randint(0, cap, (N,), generator=gen)
    pos[0], pos[-1] = P, P + cap - 1  # the first and the last slot
    # what no sequence sees may hold anything
    x["kp"][:, :, P:], x["vp"][:, :, P:] = float("nan"), float("inf")
    for n, p in enumerate(pos.tolist()):
        x["kc"][n, :, p - P + 1:], x["vc"][n, :, p - P + 1:] = float("inf"), float("nan")
    o, d = step(x, pos, P, R)
    assert swa.get_last_device_error() == (swa.OK, 0)
    ref = reference(x, pos, P, R, 1e4)
    assert torch.isfinite(o).all() and su.rel(o, ref) <= REL
    for n in ("kc", "vc"):
        assert su.neighbours(d[n].cpu(), x[n]).all()


@pytest.mark.parametrize("N,Hq,Hkv,P,pcap,cap,R", [
    (1, 1, 1, 1, 1, 1, 42), (1, 8, 1, 127, 128, 3, 42), (3, 4, 2, 128, 128, 1, 0),
    (2, 6, 2, 129, 300, 130, 32), (17, 8, 1, 640, 640, 5, 48), (32, 4, 1, 257, 257, 2, 42),
    (33, 4, 1, 1000, 1024, 9, 42), (70, 8, 2, 300, 300, 4, 42), (5, 3, 3, 2049, 2049, 33, 42),
    (4, 4, 1, 0, 16, 40, 42), (2, 2, 1, 64, 64, 2100, 42),
])
def test_shared_decode(N, Hq, Hkv, P, pcap, cap, R):
    check(N, Hq, Hkv, P, pcap, cap, R, seed=N + P)


def test_keys_far_above_the_norm_bound():
    """A cache is the caller's: scores that grow from tile to tile by more than the
    references' slack, in the order that makes every tile raise them."""
    N, Hq, Hkv, P, cap = 3, 4, 1, 1400, 4
    x = inputs(N, Hq, Hkv, P, P, cap, seed=5)
    x["kp"] = (x["kp"].float() * torch.linspace(0.1, 12, P)[None, None, :, None]).to(torch.bfloat16)
    pos = torch.tensor([P, P + 1, P + 3])
    o, _ = step(x, pos, P)
    ref = reference(x, pos, P, 42, 1e4)
    # scores up to ~500: q' of 16 bits leaves 500 x 2^-16 = 8e-3 in an exponent
    assert torch.isfinite(o).all() and su.rel(o, ref) <= REL + 8e-3


def test_bad_positions_are_skipped_and_reported():
    P, cap = 200, 8
    x = inputs(4, 4, 2, P, P, cap, seed=6)
    pos = torch.tensor([P + 2, P - 1, P + cap, P])
    out = torch.full((4, 4, 128), 3.0, dtype=torch.bfloat16, device=DEV)
    o, d = step(x, pos, P, out=out)
    assert swa.get_last_device_error()[0] == swa.ERR_INVALID_ARG
    assert (o[1:3] == 3.0).all()
    for n in ("kc", "vc"):
        assert torch.equal(d[n][1:3].cpu(), x[n][1:3])
    keep = [0, 3]
    y = {n: (t[keep] if n in ("q", "k", "v", "kc", "vc") else t) for n, t in x.items()}
    assert su.rel(o[keep], reference(y, pos[keep], P, 42, 1e4)) <= REL


def test_it_is_the_plain_step_over_the_joined_cache():
    N, Hq, Hkv, P, cap = 6, 8, 2, 500, 64
    x = inputs(N, Hq, Hkv, P, P, cap, seed=7)
    pos = P + torch.tensor([0, 1, 7, 20, 40, 63])
    o, _ = step(x, pos, P, base=1e7)
    d = {n: t.to(DEV) for n, t in x.items()}
    join = lambda a, b: torch.cat([a.expand(N, -1, -1, -1), b], 2).contiguous()
    ref = swa.global_decode_step(pos.to(DEV), d["q"], d["k"], d["v"], d["wq"], d["wk"],
                                 join(d["kp"], d["kc"]), join(d["vp"], d["vc"]))
    assert su.rel(o, ref) <= 2 * REL


def test_workspace_contents_do_not_matter_and_graph_replay():
    N, Hq, Hkv, P, cap = 40, 4, 2, 900, 16
    x = inputs(N, Hq, Hkv, P, P, cap, seed=8)
    pos = P + torch.arange(N) % cap
    n = swa.global_decode_shared_workspace_size(N, Hq, Hkv, P, cap)
    ws = torch.full((n,), 255, dtype=torch.uint8, device=DEV)
    o, d = step(x, pos, P, workspace=ws)
    dpos = pos.to(DEV)
    call = lambda: swa.global_decode_shared(dpos, d["q"], d["k"], d["v"], d["wq"], d["wk"], d["kp"],
                                            d["vp"], P, d["kc"], d["vc"], rope_base=1e4)
    assert torch.equal(call(), o)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        og = call()
    d["q"].copy_(d["q"].flip(0))
    dpos.copy_((P + (torch.arange(N) * 3) % cap).to(DEV))
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(og, call())
    assert swa.get_last_device_error() == (swa.OK, 0)


def test_forced_timeout_is_reported_and_context_survives():
    x = inputs(2, 4, 1, 300, 300, 8, seed=9)
    step(x, torch.tensor([300, 305]), 300, flags=swa.FLAG_FORCE_TIMEOUT)
    assert swa.get_last_device_error()[0] == swa.ERR_DEVICE_TIMEOUT
    check(2, 4, 1, 300, 300, 8)


def test_parallel_samples_of_one_prompt():
    """The operators together: one prompt through a window layer with sinks and a
    global layer, then three samples that share its caches, token by token, against
    forwards of the three whole sequences."""
    N, T, more, Hq, Hkv, S = 3, 300, 12, 4, 2, 4
    gen = torch.Generator().manual_seed(70)
    n = lambda *s: torch.randn(s, generator=gen).to(torch.bfloat16).to(DEV)
    w = [(1 + 0.1 * torch.randn(128, generator=gen)).to(DEV) for _ in range(2)]
    prompt = [n(1, T, h, 128) for h in (Hq, Hkv, Hkv, Hq)]
    tail = [n(N, more, h, 128) for h in (Hq, Hkv, Hkv, Hq)]
    whole = [torch.cat([p.expand(N, -1, -1, -1), t], 1).contiguous() for p, t in zip(prompt, tail)]
    o_win = swa.sink_fwd(*whole, *w, S)
    full = [torch.empty(N, Hkv, T + more, 128, dtype=torch.bfloat16, device=DEV) for _ in range(2)]
    o_glb = swa.global_fwd(*whole[:3], *w, *full)

    # the prompt once
    swa.sink_fwd(*prompt, *w, S)
    ring = [torch.empty(1, Hkv, 128, 128, dtype=torch.bfloat16, device=DEV) for _ in range(2)]
    sink = [torch.empty(1, Hkv, S, 128, dtype=torch.bfloat16, device=DEV) for _ in range(2)]
    swa.prefill_to_ring(prompt[1], prompt[2], w[1], *ring, Hq=Hq, rope_base=1e4)
    swa.prefill_to_sinks(prompt[1], prompt[2], w[1], *sink, Hq=Hq, rope_base=1e4)
    pre = [torch.empty(1, Hkv, T, 128, dtype=torch.bfloat16, device=DEV) for _ in range(2)]
    swa.global_fwd(*prompt[:3], *w, *pre)
    # forked for the samples
    ring = [c.repeat(N, 1, 1, 1) for c in ring]
    sink = [c.repeat(N, 1, 1, 1) for c in sink]
    own = [torch.empty(N, Hkv, more, 128, dtype=torch.bfloat16, device=DEV) for _ in range(2)]
    win, glb = [], []
    for i in range(more):
        pos = torch.full((N,), T + i, dtype=torch.int64, device=DEV)
        q, k, v, g = [t[:, i].contiguous() for t in tail]
        win.append(swa.sink_decode_step(pos, q, k, v, g, *w, *ring, *sink, rope_base=1e4))
        glb.append(swa.global_decode_shared(pos, q, k, v, *w, *pre, T, *own, rope_base=1e4))
    assert swa.get_last_device_error() == (swa.OK, 0)
    assert su.rel(torch.stack(win, 1), o_win[:, T:]) <= 2 * REL
    assert su.rel(torch.stack(glb, 1), o_glb[:, T:]) <= 2 * REL
