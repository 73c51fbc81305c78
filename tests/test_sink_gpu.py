"""GPU parity of sink attention (forward, backward, decode, handoff) with plain 64-bit
forms, and its behaviour at the edges: lengths, head groups, values that are not finite
in masked places, extreme magnitudes, streams, graphs, refusals.

Tolerances.  Outputs are bf16: a rounding is off by at most 2^-8 of the value, so by
3.9e-3 in the relative 2-norm whatever happens before.  The operands q', k', P, dA, dS
are fp16 (2^-12 of a value, half a step) with at most two of them in a product: their
share of a 2-norm is below 4 x 2^-12 = 1e-3.  REL = 5e-3 is the library's bar and covers
both.  dg is dO o (1 - sigmoid) from the bf16 o: two roundings, 2 x 2^-8 + 1e-3 = 8.9e-3.
Weight gradients are fp32 sums of such terms over all rows: 5e-3 as well."""
import pytest
import torch

import hybrid_sliding_window_gated_b200 as swa
import sink_testutil as su

pytestmark = pytest.mark.gpu
DEV = "cuda"
REL, REL_DG = 5e-3, 8.9e-3


def ok():
    assert swa.get_last_device_error() == (swa.OK, 0)


def forward(x, S, R=42, base=1e4, scale=0.0, **kw):
    return swa.sink_fwd(*su.args(x, DEV), S, rot_dim=R, rope_base=base, scale=scale, want_lse=True,
                        **kw)


def check_forward(x, S, R=42, base=1e4, scale=0.0):
    o, lse = forward(x, S, R, base, scale)
    ok()
    o_ref, lse_ref = su.sink_forward(*su.args(x, dtype=torch.float64), S, R, base, scale)
    assert torch.isfinite(o).all()
    assert su.rel(o, o_ref) <= REL
    # every row for itself: the same bound, with the row's own norm
    d = (o.double().cpu() - o_ref).norm(dim=-1)
    assert (d <= 2 * REL * o_ref.norm(dim=-1) + 1e-30).all()
    # a score's error is at most 2 x 2^-11 |q'||k'| scale <= 2^-10 sqrt(128) max|w|^2
    assert (lse.double().cpu() - lse_ref).abs().max() <= 0.03
    return o, lse


SHAPES = [
    # B, T, Hq, Hkv, n_sink, R
    (1, 1, 1, 1, 4, 42), (1, 2, 2, 1, 0, 42), (2, 63, 4, 2, 3, 42), (1, 64, 2, 2, 16, 0),
    (1, 65, 3, 1, 1, 32), (2, 128, 4, 4, 5, 48), (1, 129, 8, 2, 4, 42), (3, 191, 6, 2, 16, 42),
    (1, 200, 5, 1, 7, 42), (1, 257, 2, 1, 8, 42), (2, 320, 7, 1, 2, 42),
]


@pytest.mark.parametrize("B,T,Hq,Hkv,S,R", SHAPES)
def test_forward(B, T, Hq, Hkv, S, R):
    check_forward(su.draw(B, T, Hq, Hkv, seed=T + S, g_std=2.0), S, R)


def test_forward_long_positions_and_base():
    check_forward(su.draw(1, 700, 2, 1, seed=5), 4, base=1e7)


@pytest.mark.parametrize("B,T,Hq,Hkv,S", [(300, 1, 2, 1, 4), (400, 64, 1, 1, 4), (260, 65, 4, 2, 3),
                                          (150, 130, 2, 1, 16), (100, 200, 6, 3, 2)])
def test_forward_runs_that_cross_chains(B, T, Hq, Hkv, S):
    """More tiles than SMs, so one CTA walks over several sequences' ends: every copy of
    one sequence comes out as that sequence alone does, bit for bit."""
    one = su.draw(1, T, Hq, Hkv, seed=6)
    o1, l1 = check_forward(one, S)
    many = {n: (t if n in ("wq", "wk") else t.expand(B, *t.shape[1:]).contiguous())
            for n, t in one.items()}
    for _ in range(3):
        o, lse = forward(many, S)
        ok()
        assert torch.equal(o, o1.expand_as(o)) and torch.equal(lse, l1.expand_as(lse))


def test_no_sinks_is_the_window_forward():
    x = su.draw(2, 300, 4, 2, seed=7)
    o, lse = forward(x, 0)
    o2, lse2 = swa.fwd(*su.args(x, DEV), want_lse=True)
    # swa_fwd's own bar is REL too
    assert su.rel(o, o2) <= 2 * REL and (lse - lse2).abs().max() <= 0.06


def test_large_norm_weights_and_scale():
    """Scores in the hundreds: rows whose probability sits on one key."""
    x = su.draw(1, 260, 2, 1, seed=8)
    x["wq"], x["wk"] = 20 * x["wq"], 20 * x["wk"]
    o, lse = forward(x, 4)
    ok()
    o_ref, lse_ref = su.sink_forward(*su.args(x, dtype=torch.float64), 4, 42, 1e4)
    # a score's error: 2^-11 per operand of |q'||k'| scale <= sqrt(128) 20^2 1.3^2
    assert torch.isfinite(o).all()
    assert ((lse.double().cpu() - lse_ref).abs() <= 2 ** -10 * 11.4 * 400 * 1.7).all()
    # where one key holds the row (p > 1 - 1e-6) the error of the scores cannot matter
    check_forward(su.draw(1, 260, 2, 1, seed=8), 4, scale=0.5)


@pytest.mark.parametrize("factor", [1e-36, 1e-7, 1e5, 1e36])
def test_v_of_any_magnitude(factor):
    x = su.draw(1, 300, 2, 1, seed=9)
    x["v"] = (x["v"].float() * factor).to(torch.bfloat16)
    check_forward(x, 4)


def test_v_rows_of_mixed_magnitude():
    x = su.draw(1, 300, 4, 1, seed=10)
    gen = torch.Generator().manual_seed(1)
    x["v"] = (x["v"].float() * 10.0 ** torch.randint(-4, 5, (1, 300, 1, 1), generator=gen)).to(
        torch.bfloat16)
    check_forward(x, 4)


def test_tiny_v_rows_beside_ordinary_ones():
    """The rows of one warp need different scales."""
    x = su.draw(1, 300, 4, 2, seed=72)
    x["v"][0, :100] = (x["v"][0, :100].float() * 1e-30).to(torch.bfloat16)
    x["v"][0, 101:105] = (x["v"][0, 101:105].float() * 1e30).to(torch.bfloat16)
    check_forward(x, 0)


@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("inf")])
def test_values_that_are_not_finite_reach_only_rows_that_see_them(bad):
    """Rows behind a padded sequence, keys out of the window: a masked key has no part
    in a row, whatever it holds."""
    T, S = 400, 3
    x = su.draw(1, T, 4, 2, seed=11)
    clean = {n: t.clone() for n, t in x.items()}
    x["v"][0, 2, 0, 5] = bad      # a sink
    x["v"][0, 100, 1, 7] = bad    # rows 100 .. 227
    x["k"][0, 390, 1, 3] = bad    # rows 390 ..: their whole output
    x["v"][0, T - 1] = bad
    o, _ = forward(x, S)
    o_ref, _ = forward(clean, S)
    ok()
    hit = torch.zeros_like(o, dtype=torch.bool)
    hit[0, 2:, :2, 5] = True                # KV head 0: every later row sees the sink
    hit[0, 100:228, 2:, 7] = True
    hit[0, 390:, 2:] = True
    hit[0, T - 1] = True
    assert not torch.isfinite(o[hit]).any()
    assert torch.isfinite(o[~hit]).all()
    assert su.rel(o[~hit], o_ref[~hit]) <= REL


@pytest.mark.parametrize("size", [1.0, 1e-3, 1e-20])
def test_huge_values_in_masked_places(size):
    """Keys that a row does not see leave its V rows' scale alone: later tokens, and
    those that the window has left behind."""
    x = su.draw(1, 400, 4, 2, seed=71)
    x["v"] = (x["v"].float() * size).to(torch.bfloat16)
    clean = {n: t.clone() for n, t in x.items()}
    x["v"][0, 100] = 3e38
    x["v"][0, 333:] = -3e38
    rows = torch.tensor([i for i in range(333) if i < 100 or i >= 228])
    o, _ = forward(x, 3)
    o_ref, _ = su.sink_forward(*su.args(clean, dtype=torch.float64), 3, 42, 1e4)
    assert torch.isfinite(o).all()
    d = (o.double().cpu() - o_ref)[:, rows].norm(dim=-1)
    assert (d <= 2 * REL * o_ref[:, rows].norm(dim=-1)).all()


def test_gate_at_infinity():
    x = su.draw(1, 200, 2, 1, seed=12)
    x["g"][0, :, 0] = -float("inf")
    o, _ = forward(x, 4)
    assert (o[0, :, 0] == 0).all() and torch.isfinite(o).all()


# ------------------------------------------------------------------ backward


def check_backward(x, S, R=42, base=1e4, scale=0.0, names=su.NAMES):
    t = su.args(x, DEV)
    kw = dict(rot_dim=R, rope_base=base, scale=scale)
    o, lse = swa.sink_fwd(*t, S, want_lse=True, **kw)
    grads = swa.sink_bwd(*t, o, lse, x["dO"].to(DEV), S, **kw)
    ok()
    ref = su.sink_gradients(su.args(x), x["dO"], S, R, base, scale)
    # dq and dk of a sequence's first token vanish: differences against the largest
    # gradient of their kind, the rest in the 2-norm
    for name, got, want in zip(su.NAMES, grads, ref):
        assert torch.isfinite(got).all(), name
        if name in names:
            assert su.rel(got, want) <= (REL_DG if name == "g" else REL), name
    return grads


@pytest.mark.parametrize("B,T,Hq,Hkv,S,R", [s for s in SHAPES if s[1] > 1])
def test_backward(B, T, Hq, Hkv, S, R):
    check_backward(su.draw(B, T, Hq, Hkv, seed=2 * T + S, grad=True), S, R)


def test_backward_of_one_token():
    """P = 1: dq, dk, dwq and dwk vanish, dv = dA."""
    x = su.draw(2, 1, 4, 2, seed=13, grad=True)
    grads = check_backward(x, 4, names=("v", "g"))
    size = x["dO"].float().norm()
    for i in (0, 1, 4, 5):
        # dP - D of fp16 operands: 2^-11 of |dA||v| at most
        assert grads[i].float().norm().cpu() <= 2 ** -8 * size


@pytest.mark.parametrize("factor", [1e-20, 1e-6, 1e6])
def test_backward_of_gradients_of_any_magnitude(factor):
    x = su.draw(1, 200, 4, 2, seed=14, grad=True)
    x["dO"] = (x["dO"].float() * factor).to(torch.bfloat16)
    check_backward(x, 3)


@pytest.mark.parametrize("factor", [1e-33, 1e-6, 1e6, 1e33])
def test_backward_of_v_of_any_magnitude(factor):
    x = su.draw(1, 200, 2, 1, seed=15, grad=True)
    x["v"] = (x["v"].float() * factor).to(torch.bfloat16)
    check_backward(x, 3)


def test_backward_rows_without_gradient_and_shut_gates():
    x = su.draw(1, 300, 4, 2, seed=16, grad=True)
    x["dO"][0, 100:180] = 0
    x["g"][0, 200:220, 1] = -30.0
    check_backward(x, 4)


def test_backward_adds_into_weight_gradients_and_repeats_bit_for_bit():
    x = su.draw(2, 333, 4, 2, seed=17, grad=True)
    t, dO = su.args(x, DEV), x["dO"].to(DEV)
    o, lse = swa.sink_fwd(*t, 4, want_lse=True)
    a = swa.sink_bwd(*t, o, lse, dO, 4)
    ws = torch.full((swa.sink_bwd_workspace_size(2, 333, 4, 2, 4),), 255, dtype=torch.uint8,
                    device=DEV)  # NaN patterns: nothing of it may matter
    g = [torch.empty_like(y) for y in a[:4]] + [torch.ones_like(a[4]), 2 * torch.ones_like(a[5])]
    swa.sink_bwd(*t, o, lse, dO, 4, workspace=ws, grads=tuple(g))
    ok()
    for y, z in zip(a[:4], g[:4]):
        assert torch.equal(y, z)
    assert torch.equal(g[4], a[4] + 1) and torch.equal(g[5], a[5] + 2)


def test_sequences_of_a_batch_do_not_touch_each_other():
    x = su.draw(3, 150, 4, 1, seed=18, grad=True)
    t, dO = su.args(x, DEV), x["dO"].to(DEV)
    o, lse = swa.sink_fwd(*t, 4, want_lse=True)
    whole = swa.sink_bwd(*t, o, lse, dO, 4)
    for b in range(3):
        s = [y[b:b + 1].contiguous() for y in t[:4]] + t[4:]
        ob, lb = swa.sink_fwd(*s, 4, want_lse=True)
        assert torch.equal(ob[0], o[b]) and torch.equal(lb[0], lse[b])
        part = swa.sink_bwd(*s, ob, lb, dO[b:b + 1].contiguous(), 4)
        for y, z in zip(part[:4], whole[:4]):
            assert torch.equal(y[0], z[b])


# -------------------------------------------------------------------- decode


def decode_ref(pos, q, k, v, g, wq, wk, kc, vc, ks, vs, R, base):
    """o of one step in 64 bits; the caches (bf16, CPU) are updated as it defines."""
    N, Hq, _ = q.shape
    S = ks.shape[2]
    qq = su.norm_rope(q.double(), wq.double(), pos, R, base)
    kk = su.norm_rope(k.double(), wk.double(), pos, R, base).to(torch.bfloat16)
    out = torch.empty(q.shape, dtype=torch.float64)
    for n, p in enumerate(pos.tolist()):
        kc[n, :, p % 128], vc[n, :, p % 128] = kk[n], v[n]
        if p < S:
            ks[n, :, p], vs[n, :, p] = kk[n], v[n]
        early = max(0, min(S, p - 127))
        held = [t % 128 for t in range(max(0, p - 127), p + 1)]
        ctx = lambda a, b: torch.cat([b[n, :, :early], a[n][:, held]], 1).double()
        out[n] = su.context_attention(qq[n], ctx(kc, ks), ctx(vc, vs)) * torch.sigmoid(g[n].double())
    return out


def decode_inputs(N, Hq, Hkv, S, seed):
    gen = torch.Generator().manual_seed(seed)
    n = lambda *s: torch.randn(s, generator=gen).to(torch.bfloat16)
    x = [n(N, Hq, 128), n(N, Hkv, 128), n(N, Hkv, 128), n(N, Hq, 128),
         1 + 0.1 * torch.randn(128, generator=gen), 1 + 0.1 * torch.randn(128, generator=gen)]
    caches = [n(N, Hkv, 128, 128), n(N, Hkv, 128, 128), n(N, Hkv, S, 128), n(N, Hkv, S, 128)]
    return x, caches


@pytest.mark.parametrize("Hq,Hkv,S,R", [(4, 1, 4, 42), (8, 1, 16, 42), (3, 3, 1, 0), (12, 2, 9, 32),
                                        (10, 5, 8, 48), (2, 1, 0, 42)])
def test_decode(Hq, Hkv, S, R):
    pos = torch.tensor([0, 1, S, 15, 16, 127, 128, 128 + S, 143, 144, 300, 262143])
    x, caches = decode_inputs(len(pos), Hq, Hkv, S, seed=20 + S)
    # slots that hold no token may hold anything
    for n, p in enumerate(pos.tolist()):
        for c in caches[:2]:
            if p < 127:
                c[n, :, p + 1:] = float("nan")
        for c in caches[2:]:
            c[n, :, max(0, min(S, p - 127)):] = float("inf")
    dev = [c.to(DEV) for c in caches]
    o = swa.sink_decode_step(pos.to(DEV), *[y.to(DEV) for y in x], *dev, rot_dim=R, rope_base=1e4)
    ok()
    ref = decode_ref(pos, *x, *caches, R, 1e4)
    assert torch.isfinite(o).all() and su.rel(o, ref) <= REL
    for got, want in zip(dev, caches):
        got = got.cpu()
        same = got.view(torch.int16) == want.view(torch.int16)
        assert su.neighbours(got, want).all() and (~same).sum() <= 1e-3 * same.numel()


def test_decode_bad_position_is_skipped_and_reported():
    x, caches = decode_inputs(3, 4, 2, 4, seed=30)
    dev = [c.to(DEV) for c in caches]
    o = torch.full((3, 4, 128), 3.0, dtype=torch.bfloat16, device=DEV)
    swa.sink_decode_step(torch.tensor([5, -1, 200]).to(DEV), *[y.to(DEV) for y in x], *dev, out=o)
    assert swa.get_last_device_error()[0] == swa.ERR_INVALID_ARG
    ok()
    assert (o[1] == 3.0).all() and (o[0] != 3.0).any() and (o[2] != 3.0).any()
    for c, d in zip(caches, dev):
        assert torch.equal(d[1].cpu(), c[1])


@pytest.mark.parametrize("T,S", [(1, 4), (100, 16), (260, 4)])
def test_prefill_handoff_and_decode_continue_the_sequence(T, S):
    """Prefill, handoff to rings and sinks, then token by token: the rows of one long
    forward."""
    more, Hq, Hkv = 150, 4, 2
    x = su.draw(2, T + more, Hq, Hkv, seed=40 + T)
    t = su.args(x, DEV)
    o_all = swa.sink_fwd(*t, S)
    head = [y[:, :T].contiguous() for y in t[:4]]
    assert torch.equal(swa.sink_fwd(*head, *t[4:], S), o_all[:, :T])
    kc = torch.full((2, Hkv, 128, 128), float("nan"), dtype=torch.bfloat16, device=DEV)
    vc = kc.clone()
    ks = torch.full((2, Hkv, S, 128), float("nan"), dtype=torch.bfloat16, device=DEV)
    vs = ks.clone()
    swa.prefill_to_ring(head[1], head[2], t[5], kc, vc, Hq=Hq, rope_base=1e4)
    swa.prefill_to_sinks(head[1], head[2], t[5], ks, vs, Hq=Hq, rope_base=1e4)
    outs = []
    for i in range(T, T + more):
        pos = torch.full((2,), i, dtype=torch.int64, device=DEV)
        outs.append(swa.sink_decode_step(pos, *[y[:, i].contiguous() for y in t[:4]], *t[4:], kc, vc,
                                         ks, vs, rope_base=1e4))
    ok()
    # the decode's k' is bf16: 2^-8 of a key more in the scores, and both outputs' roundings
    assert su.rel(torch.stack(outs, 1), o_all[:, T:]) <= 2 * REL


def test_sinks_of_a_ragged_batch_and_bad_lengths():
    Hkv, S = 2, 6
    gen = torch.Generator().manual_seed(50)
    k = torch.randn(40, Hkv, 128, generator=gen).to(torch.bfloat16).to(DEV)
    v = torch.randn(40, Hkv, 128, generator=gen).to(torch.bfloat16).to(DEV)
    wk = (1 + 0.1 * torch.randn(128, generator=gen)).to(DEV)
    i64 = lambda *a: torch.tensor(a, dtype=torch.int64, device=DEV)
    starts, lens, pos0 = i64(0, 3, 20, 39, 30, 5), i64(3, 17, 10, 2, 10, 0), i64(0, 0, 4, 0, -1, 0)
    ks = torch.full((6, Hkv, S, 128), 7.0, dtype=torch.bfloat16, device=DEV)
    vs = ks.clone()
    swa.prefill_to_sinks(k, v, wk, ks, vs, starts, lens, pos0, Hq=4, rope_base=1e4)
    assert swa.get_last_device_error()[0] == swa.ERR_INVALID_ARG  # sequences 3 and 4
    reach = {0: range(0, 3), 1: range(0, 6), 2: range(4, 6), 3: (), 4: (), 5: ()}
    for b, slots in reach.items():
        for s in range(S):
            if s in slots:
                row = int(starts[b]) + s - int(pos0[b])
                want = su.norm_rope(k[row].double().cpu(), wk.double().cpu(), torch.tensor(s), 42, 1e4)
                assert su.rel(ks[b, :, s], want) <= 2 ** -8
                assert torch.equal(vs[b, :, s], v[row])
            else:
                assert (ks[b, :, s] == 7).all() and (vs[b, :, s] == 7).all()


# ------------------------------------------------- streams, graphs, failures


def test_other_streams_and_graph_replay():
    x = su.draw(1, 300, 4, 2, seed=60, grad=True)
    t, dO = su.args(x, DEV), x["dO"].to(DEV)
    o, lse = swa.sink_fwd(*t, 4, want_lse=True)
    want = swa.sink_bwd(*t, o, lse, dO, 4)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    got = []
    for s in streams:  # two at once, each with its own workspace
        with torch.cuda.stream(s):
            o2, l2 = swa.sink_fwd(*t, 4, want_lse=True)
            got.append(swa.sink_bwd(*t, o2, l2, dO, 4))
    torch.cuda.synchronize()
    for g in got:
        assert all(torch.equal(a, b) for a, b in zip(g, want))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        o3, l3 = swa.sink_fwd(*t, 4, want_lse=True)
        g3 = swa.sink_bwd(*t, o3, l3, dO, 4)
    y = su.draw(1, 300, 4, 2, seed=61, grad=True)
    for a, n in zip(t, su.NAMES):
        a.copy_(y[n])
    dO.copy_(y["dO"])
    for _ in range(2):
        graph.replay()
    torch.cuda.synchronize()
    o4, l4 = swa.sink_fwd(*t, 4, want_lse=True)
    g4 = swa.sink_bwd(*t, o4, l4, dO, 4)
    assert torch.equal(o3, o4) and torch.equal(l3, l4)
    assert all(torch.equal(a, b) for a, b in zip(g3, g4))
    ok()


def test_forced_timeout_is_reported_and_context_survives():
    x = su.draw(1, 200, 2, 1, seed=62)
    forward(x, 4, flags=swa.FLAG_FORCE_TIMEOUT)
    assert swa.get_last_device_error()[0] == swa.ERR_DEVICE_TIMEOUT
    y, caches = decode_inputs(2, 2, 1, 4, seed=63)
    swa.sink_decode_step(torch.tensor([3, 200]).to(DEV), *[z.to(DEV) for z in y],
                         *[c.to(DEV) for c in caches], flags=swa.FLAG_FORCE_TIMEOUT)
    assert swa.get_last_device_error()[0] == swa.ERR_DEVICE_TIMEOUT
    check_forward(x, 4)
