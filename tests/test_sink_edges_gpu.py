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


# ------------------------------------------------------------------ eps = 0


def cancelled(x, S):
    """What fp16 dP costs dq, as a bound on its 2-norm over all rows (64 bits).  dS = P (dP - D)
    cancels where a row's probability sits on few keys, as in a sequence's first tokens: dP
    is off by 2^-11 of itself, so dq' by scale 2^-11 sum_j P |dP| |k'|, and RoPE and the norm
    pass on at most max|w| / rms of that."""
    q, k, v, g, wq, wk = su.args(x, dtype=torch.float64)
    B, T, Hq, _ = q.shape
    Hkv = k.shape[2]
    G = Hq // Hkv
    pos = torch.arange(T).expand(B, T)
    qq, kk = su.norm_rope(q, wq, pos, 42, 1e4), su.norm_rope(k, wk, pos, 42, 1e4)
    dA = x["dO"].double() * torch.sigmoid(g)
    total = 0.0
    for i in range(T):
        js = su.visible(i, S, T)
        heads = lambda y: y[:, i].reshape(B, Hkv, G, 128)
        p = torch.softmax(torch.einsum("bhgd,bjhd->bhgj", heads(qq), kk[:, js]) / math.sqrt(128), -1)
        dp = torch.einsum("bhgd,bjhd->bhgj", heads(dA), v[:, js])
        size = kk[:, js].norm(dim=-1).permute(0, 2, 1)[:, :, None]
        e = 2.0 ** -11 / math.sqrt(128) * (p * dp.abs() * size).sum(-1)
        rms = heads(q).pow(2).mean(-1).sqrt()
        total += float((e * wq.abs().max() / rms).pow(2).sum())
    return math.sqrt(total)


@pytest.mark.parametrize("B,T,Hq,Hkv,S", [(1, 2, 2, 1, 4), (2, 65, 4, 2, 3), (1, 200, 3, 1, 16),
                                          (1, 64, 2, 2, 0)])
def test_backward_without_eps(B, T, Hq, Hkv, S):
    """Tokens that only fill up the last tile have no norm: they take no part.  The 64-bit
    form's eps of 1e-6 is a factor of 1 - 5e-7 on rows of mean square 1."""
    x = su.draw(B, T, Hq, Hkv, seed=110 + T, grad=True)
    t = su.args(x, DEV)
    o, lse = swa.sink_fwd(*t, S, want_lse=True, eps=0.0)
    grads = swa.sink_bwd(*t, o, lse, x["dO"].to(DEV), S, eps=0.0)
    ok()
    for name, got, want in zip(su.NAMES, grads, su.sink_gradients(su.args(x), x["dO"], S, 42, 1e4)):
        assert torch.isfinite(got).all(), name
        bound = REL_DG if name == "g" else REL
        if name == "q":
            bound += cancelled(x, S) / float(want.norm())
        if name == "wq":  # sums of u RoPE^-1(dq') with |u| <= 4 and rows' errors of either sign
            bound += 4 * cancelled(x, S) / float(want.norm())
        assert su.rel(got, want) <= bound, name


# ------------------------------------------------- magnitudes at bf16's ends


@pytest.mark.parametrize("T,v,dO", [(200, 3e38, 1e-3), (70, 3e38, 1e-3), (200, 1.2e38, 1e-30),
                                    (200, 1e-2, 1.2e38), (333, 3e38, 1e-34)])
def test_backward_of_the_largest_values(T, v, dO):
    """v or dO up to the end of bf16's range where the gradients themselves are finite."""
    x = su.draw(1, T, 2, 1, seed=120, grad=True)
    gen = torch.Generator().manual_seed(121)
    for name, top in (("v", v), ("dO", dO)):
        sign = 2.0 * torch.randint(0, 2, x[name].shape, generator=gen) - 1.0
        size = 0.25 + 0.75 * torch.rand(x[name].shape, generator=gen)
        x[name] = (sign * size * top).to(torch.bfloat16)
    ref = su.sink_gradients(su.args(x), x["dO"], 3, 42, 1e4)
    assert max(float(r.abs().max()) for r in ref) < 3e38
    check_backward(x, 3)


# -------------------------------------- values that are not finite, backward


@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("inf")])
@pytest.mark.parametrize("where", ["k", "k_late", "v", "v_sink", "q", "dO"])
def test_backward_hides_what_is_masked(where, bad):
    """A row that is not finite reaches the gradients of the rows that a visible pair
    joins it with, and no others.  Token 10 is no sink, though it shares the sinks' tile."""
    T, S, Hq, Hkv = 400, 3, 4, 2
    x = su.draw(1, T, Hq, Hkv, seed=130, grad=True)
    clean = {n: t.clone() for n, t in x.items()}
    name, at, head = {"k": ("k", 10, 0), "k_late": ("k", 390, 1), "v": ("v", 100, 1),
                      "v_sink": ("v", 2, 0), "q": ("q", 300, 1), "dO": ("dO", 250, 2)}[where]
    x[name][0, at, head, 5] = bad
    t, dO = su.args(x, DEV), x["dO"].to(DEV)
    o, lse = swa.sink_fwd(*t, S, want_lse=True)
    got = swa.sink_bwd(*t, o, lse, dO, S)
    ok()
    want = su.sink_gradients(su.args(clean), clean["dO"], S, 42, 1e4)
    # queries (by query head) whose probabilities or dP the row enters, then the keys they see
    kvh = head if name in ("k", "v") else head // (Hq // Hkv)
    heads = range(2 * kvh, 2 * kvh + 2) if name in ("k", "v") else [head]
    queries = [i for i in range(T) if at in su.visible(i, S, T)] if name in ("k", "v") else [at]
    keys = sorted({j for i in queries for j in su.visible(i, S, T)})
    free = {n: torch.ones_like(x[n], dtype=torch.bool) for n in ("q", "k", "v", "g")}
    for h in heads:
        free["q"][0, queries, h] = False
        free["g"][0, queries, h] = False
    for n in ("k", "v"):
        free[n][0, keys, kvh] = False
    for n, y, ref in zip("qkvg", got, want):
        f = free[n]
        assert torch.isfinite(y[f.to(DEV)]).all(), n
        assert su.rel(y.cpu()[f], ref[f]) <= (REL_DG if n == "g" else REL), n
    # what a visible pair joins with it is not quietly finite
    for h in heads:
        assert (~torch.isfinite(got[0][0, queries, h])).any(dim=-1).all()
    assert (~torch.isfinite(got[1][0, keys, kvh])).any(dim=-1).all()


# ---------------------------------------- V entries far below their row's own


@pytest.mark.parametrize("top", [2.0 ** -6, 1.0, 100.0, 127.0, 3e4, 1e10])
def test_forward_keeps_small_dims_of_v(top):
    """Every dim of o by itself, where V's dims differ by up to 2^19 in size: an entry keeps
    its bf16 bits whatever its row's largest is.  P is off by 2^-11 of an entry, which the
    bound of a whole row covers for each dim as well."""
    x = su.draw(1, 300, 2, 1, seed=140)
    size = top * 2.0 ** (-19.0 * torch.arange(128) / 127)
    gen = torch.Generator().manual_seed(141)
    sign = 2.0 * torch.randint(0, 2, (1, 300, 1, 128), generator=gen) - 1.0
    x["v"] = (sign * size * (0.75 + 0.25 * torch.rand(1, 300, 1, 128, generator=gen))).to(
        torch.bfloat16)
    x["v"][..., 0] = (sign[..., 0] * top).to(torch.bfloat16)
    o, _ = forward(x, 4)
    ok()
    o_ref, _ = su.sink_forward(*su.args(x, dtype=torch.float64), 4, 42, 1e4)
    d = (o.double().cpu() - o_ref).norm(dim=1) / o_ref.norm(dim=1)
    assert d.max() <= REL, d.max()


@pytest.mark.parametrize("big", [1.0, 1e32, 1e36, 2e38])
@pytest.mark.parametrize("around", [1.0, 1e-30, 1e10])
def test_forward_finite_dims_beside_an_infinity(big, around):
    """A visible V row with one infinite entry and others of any size: the other dims of the
    rows that see it come out as the 64-bit form's."""
    x = su.draw(1, 300, 2, 1, seed=142)
    x["v"] = (x["v"].float() * around).to(torch.bfloat16)
    x["v"][0, 100, 0, 5] = float("inf")
    x["v"][0, 100, 0, 8:24] = big
    o, _ = forward(x, 4)
    ok()
    o_ref, _ = su.sink_forward(*su.args(x, dtype=torch.float64), 4, 42, 1e4)
    dims = [d for d in range(128) if d != 5]
    got, want = o.double().cpu()[0, 100:228], o_ref[0, 100:228]
    assert not torch.isfinite(got[..., 5]).any()
    assert torch.isfinite(got[..., dims]).all()
    for part in (range(8, 24), [d for d in dims if not 8 <= d < 24]):
        d = (got - want)[..., part].norm(dim=-1)
        assert (d <= 2 * REL * want[..., part].norm(dim=-1)).all()


# ----------------------------------------- the backward's other launch shapes


def gathered_forward(q, k, v, g, wq, wk, n_sink, R=42, base=1e4):
    """su.sink_forward for one sequence, each query's keys gathered at once (64 bits)."""
    T, Hq, Hkv = q.shape[1], q.shape[2], k.shape[2]
    dev, n_sink = q.device, min(n_sink, q.shape[1])
    cpu = lambda y, w: su.norm_rope(y.cpu(), w.cpu(), torch.arange(T).expand(1, T), R, base).to(dev)
    qq, kk = cpu(q, wq)[0].reshape(T, Hkv, -1, 128), cpu(k, wk)[0]
    i = torch.arange(T, device=dev)
    idx = torch.cat([i[:, None] - torch.arange(127, -1, -1, device=dev),
                     torch.arange(n_sink, device=dev).expand(T, n_sink)], 1)
    seen = torch.cat([idx[:, :128] >= 0, idx[:, 128:] <= i[:, None] - 128], 1)
    idx = idx.clamp_min(0)
    s = torch.einsum("thgd,tjhd->thgj", qq, kk[idx]) / math.sqrt(128)
    p = torch.softmax(s.masked_fill(~seen[:, None, None], -math.inf), -1)
    a = torch.einsum("thgj,tjhd->thgd", p, v[0][idx]).reshape(1, T, Hq, 128)
    return a * torch.sigmoid(g)


def gathered_gradients(x, n_sink):
    t = [y.double().to(DEV).requires_grad_() for y in su.args(x)]
    o = gathered_forward(*t, n_sink)
    return torch.autograd.grad((o * x["dO"].double().to(DEV)).sum(), t)


def test_gathered_form_is_the_plain_one():
    x = su.draw(1, 300, 4, 2, seed=150, grad=True)
    for a, b in zip(gathered_gradients(x, 5), su.sink_gradients(su.args(x), x["dO"], 5, 42, 1e4)):
        assert su.rel(a, b) <= 1e-12


@pytest.mark.parametrize("T,Hq,Hkv,S", [(4200, 2, 1, 4), (5000, 3, 1, 16), (4097, 4, 2, 0)])
def test_backward_of_long_sequences(T, Hq, Hkv, S):
    """More than 4,096 tokens: the sinks' pass in longer chunks."""
    x = su.draw(1, T, Hq, Hkv, seed=151 + T, grad=True)
    t = su.args(x, DEV)
    o, lse = swa.sink_fwd(*t, S, want_lse=True)
    grads = swa.sink_bwd(*t, o, lse, x["dO"].to(DEV), S)
    ok()
    for name, got, want in zip(su.NAMES, grads, gathered_gradients(x, S)):
        assert su.rel(got, want) <= (REL_DG if name == "g" else REL), name


@pytest.mark.parametrize("B,T,Hq,Hkv,S", [(150, 130, 4, 1, 4), (110, 130, 8, 1, 3),
                                          (33, 130, 5, 1, 4), (20, 200, 7, 1, 16),
                                          (30, 65, 10, 2, 2)])
def test_backward_of_many_sequences(B, T, Hq, Hkv, S):
    """From one head per CTA of the query-major pass to all of a group in one, and uneven
    parts between: copies of one sequence get its gradients, dwq and dwk B times its own."""
    one = su.draw(1, T, Hq, Hkv, seed=160 + B, grad=True)
    single = check_backward(one, S)
    rep = lambda y: y.expand(B, *y.shape[1:]).contiguous()
    x = {n: (y if n in ("wq", "wk") else rep(y)) for n, y in one.items()}
    t = su.args(x, DEV)
    o, lse = swa.sink_fwd(*t, S, want_lse=True)
    grads = swa.sink_bwd(*t, o, lse, x["dO"].to(DEV), S)
    ok()
    for a, b in zip(grads[:4], single[:4]):
        assert torch.equal(a, b.expand_as(a))
    for a, b in zip(grads[4:], single[4:]):
        # fp32 sums of at most B x 4 x 128 x 10 terms, 2^-24 each, of random signs
        assert su.rel(a, B * b.double()) <= 1e-4


# -------------------------------------------------------- large norm weights


def test_rows_on_one_key_with_large_norm_weights():
    """Scores in the hundreds.  Each is off by at most e = 2^-10 x 11.4 x 400 x 1.7 = 7.6,
    so keys that hold 1e-12 of a row together hold at most 1e-12 exp(2 e) = 4e-6 of it."""
    x = su.draw(1, 260, 2, 1, seed=8)
    x["wq"], x["wk"] = 20 * x["wq"], 20 * x["wk"]
    o, _ = forward(x, 4)
    ok()
    t = su.args(x, dtype=torch.float64)
    o_ref, lse = su.sink_forward(*t, 4, 42, 1e4)
    pos = torch.arange(260).expand(1, 260)
    q, k = su.norm_rope(t[0], t[4], pos, 42, 1e4)[0], su.norm_rope(t[1], t[5], pos, 42, 1e4)[0, :, 0]
    rows = 0
    for i in range(260):
        s = torch.einsum("hd,jd->hj", q[i], k[su.visible(i, 4, 260)]) / math.sqrt(128)
        p = torch.exp(s - lse[0, :, i, None])
        for h in range(2):
            top = int(p[h].argmax())
            rest = float(p[h].sum() - p[h, top])
            if rest > 1e-12:
                continue
            rows += 1
            d = (o[0, i, h].double().cpu() - o_ref[0, i, h]).norm()
            assert d <= REL * o_ref[0, i, h].norm()
    assert rows >= 200


def test_backward_with_large_norm_weights():
    """Weights of 3: a score of standard deviation 9 carries the roundings of 128 products
    of fp16 operands, of about 2e-4 each, so 9 x sqrt(2) x 2e-4 = 2.5e-3, a factor of as
    much on P and as much again on D: 5e-3 beside REL."""
    x = su.draw(1, 260, 4, 2, seed=170, grad=True)
    x["wq"], x["wk"] = 3 * x["wq"], 3 * x["wk"]
    t = su.args(x, DEV)
    o, lse = swa.sink_fwd(*t, 4, want_lse=True)
    grads = swa.sink_bwd(*t, o, lse, x["dO"].to(DEV), 4)
    ok()
    ref = su.sink_gradients(su.args(x), x["dO"], 4, 42, 1e4)
    for name, got, want in zip(su.NAMES, grads, ref):
        assert su.rel(got, want) <= REL + 5e-3, name


# ------------------------------------------------------- waits that run out


def test_backward_forced_timeout_is_reported_and_context_survives():
    x = su.draw(1, 200, 2, 1, seed=180, grad=True)
    t, dO = su.args(x, DEV), x["dO"].to(DEV)
    o, lse = swa.sink_fwd(*t, 4, want_lse=True)
    swa.sink_bwd(*t, o, lse, dO, 4, flags=swa.FLAG_FORCE_TIMEOUT)
    assert swa.get_last_device_error()[0] == swa.ERR_DEVICE_TIMEOUT
    check_backward(x, 4)
    check_forward(x, 4)


# ------------------------------------------------------- no sink caches


def test_decode_without_sink_caches_is_the_step_with_empty_ones():
    y, caches = decode_inputs(5, 4, 2, 0, seed=190)
    y, caches = [z.to(DEV) for z in y], [c.to(DEV) for c in caches]
    pos = torch.tensor([0, 3, 127, 128, 1000], device=DEV)
    rings = [c.clone() for c in caches[:2]]
    want = swa.sink_decode_step(pos, *y, *caches)
    assert torch.equal(swa.sink_decode_step(pos, *y, *rings, None, None), want)
    assert all(torch.equal(a, b) for a, b in zip(rings, caches))
    ok()


# ------------------------------------------- probabilities on few keys


@pytest.mark.parametrize("T", [2, 3, 4])
@pytest.mark.parametrize("seed", [112, 200, 201, 202, 203, 204])
def test_backward_of_a_few_tokens(T, seed):
    """dS = P (dP - D) cancels where a row's probability sits on few keys: the difference,
    not dP, is what fp16 rounds, so the bar of every other shape holds here."""
    check_backward(su.draw(1, T, 2, 1, seed=seed, grad=True), 4)


# --------------------------------------------- streams that are not torch's


class RawStream:
    def __init__(self, pointer):
        self.cuda_stream = pointer


@pytest.mark.parametrize("name", ["sink_bwd", "global_decode_shared", "fwd"])
def test_streams_of_other_libraries(name):
    """An object with a raw stream pointer, the legacy default stream among them."""
    call = calls()[name]
    want = [y.clone() for y in outputs(call(None))]
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    for pointer in (s.cuda_stream, 0):
        got = outputs(call(RawStream(pointer)))
        torch.cuda.synchronize()
        same(name, got, want)
    ok()


def test_stream_argument_in_a_captured_graph():
    t, dO = training(seed=210)
    o, lse = swa.sink_fwd(*t, 4, want_lse=True)
    want = swa.sink_bwd(*t, o, lse, dO, 4)
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        o2, l2 = swa.sink_fwd(*t, 4, want_lse=True, stream=s)
        got = swa.sink_bwd(*t, o2, l2, dO, 4, stream=s)
    for _ in range(2):
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(o2, o) and all(torch.equal(a, b) for a, b in zip(got, want))
    ok()
