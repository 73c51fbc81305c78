"""Measured cases of two operators of the hybrid attention stack.

``sink``: the gated sliding-window attention of the window layers with the
first ``n_sink`` tokens of every sequence visible to every later one: query i
attends key j when j <= i and (i - j < 128 or j < n_sink).  QK-RMSNorm, partial
RoPE at the absolute positions, GQA and the sigmoid output gate as in the
window layers.  Three kinds of call: ``prefill`` (forward), ``train`` (forward
and backward) and ``decode`` (one token per sequence over a 128-slot ring and
a small cache of the sinks).

``shared``: one decode step of a global layer for a batch of sequences that
continue one common prompt.  The prompt's K' and V lie in one cache for all of
them, each sequence's own tokens in a cache of its own.

``run`` computes the operators from elementary torch operations in fp32 (the
rotation angles in fp64), or, where ``own`` is set, through the package.
"""
import math

import torch

own = False

D = 128         # head dimension
W = 128         # window of the window layers
EPS = 1e-6


def listed():
    return [
        # the smallest prompt: a chat turn of one short sequence, few heads (latency)
        dict(name="prefill 1x256", kind="prefill", B=1, T=256, Hq=4, Hkv=1, n_sink=4, rot=42, base=1e4, g_std=1.0),
        # a batch of ordinary prompts through one layer of the model
        dict(name="prefill 4x4096", kind="prefill", B=4, T=4096, Hq=32, Hkv=8, n_sink=4, rot=42, base=1e4, g_std=2.0),
        # prompts padded to an odd length, another head layout, the most sinks
        dict(name="prefill 3x1777", kind="prefill", B=3, T=1777, Hq=24, Hkv=8, n_sink=16, rot=32, base=1e4, g_std=1.0),
        # the long-context prompt of the 256K stage
        dict(name="prefill 1x262144", kind="prefill", B=1, T=262144, Hq=32, Hkv=8, n_sink=4, rot=42, base=1e7, g_std=2.0),
        # one layer's training step at the 16K stage
        dict(name="train 1x16384", kind="train", B=1, T=16384, Hq=32, Hkv=8, n_sink=4, rot=42, base=1e4, g_std=1.0),
        # a training step on short, odd sequences and fewer heads
        dict(name="train 2x1001", kind="train", B=2, T=1001, Hq=8, Hkv=2, n_sink=1, rot=48, base=1e4, g_std=1.0),
        # one layer of a full serving batch
        dict(name="decode 256", kind="decode", N=256, Hq=32, Hkv=8, n_sink=4, rot=42, base=1e7, lo=128, hi=262144),
        # a single user's token, early and late positions (latency)
        dict(name="decode 3", kind="decode", N=3, Hq=32, Hkv=8, n_sink=16, rot=42, base=1e7, lo=0, hi=1000),
        # parallel samples of one 32K prompt (rewards, self-consistency)
        dict(name="shared 64 x 32768", kind="shared", N=64, Hq=32, Hkv=8, prefix=32768, cap=2048, rot=42, base=1e7),
        # many requests behind one very long system prompt or repository
        dict(name="shared 256 x 131072", kind="shared", N=256, Hq=32, Hkv=8, prefix=131072, cap=512, rot=42, base=1e7),
        # a few candidates of an agent's odd-sized context
        dict(name="shared 5 x 8191", kind="shared", N=5, Hq=32, Hkv=8, prefix=8191, cap=1024, rot=42, base=1e7),
        # one sequence behind a cached prompt
        dict(name="shared 1 x 2048", kind="shared", N=1, Hq=8, Hkv=2, prefix=2048, cap=256, rot=42, base=1e4),
    ]


def draw(rng):
    def log(lo, hi):
        return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))

    kind = rng.choice(["prefill", "train", "decode", "shared"])
    Hkv = rng.choice([1, 2, 4, 8])
    heads = dict(Hq=Hkv * rng.choice([1, 2, 3, 4, 8]), Hkv=Hkv, rot=rng.choice([0, 32, 42, 48]),
                 base=rng.choice([1e4, 1e7]))
    if kind == "prefill":
        T, B = log(1, 60000), rng.choice([1, 1, 2, 3, 4])
        return dict(kind=kind, B=B, T=max(1, T // B), n_sink=rng.randint(0, 16),
                    g_std=rng.choice([1.0, 2.0]), **heads)
    if kind == "train":
        # from two tokens: the gradients of q and k of a single one are zero
        T, B = log(2, 8000), rng.choice([1, 1, 2, 3])
        return dict(kind=kind, B=B, T=max(2, T // B), n_sink=rng.randint(0, 16), g_std=1.0, **heads)
    if kind == "decode":
        lo = rng.choice([0, 128])
        return dict(kind=kind, N=log(1, 256), n_sink=rng.randint(0, 16), lo=lo,
                    hi=lo + log(2, 260000), **heads)
    return dict(kind=kind, N=log(1, 256), prefix=log(1, 60000), cap=log(1, 2048), **heads)


# ------------------------------------------------------------------ inputs


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)

    def normal(*shape, std=1.0):
        x = torch.randn(shape, generator=gen, device="cuda", dtype=torch.float32)
        return (x.mul_(std) if std != 1.0 else x).to(torch.bfloat16)

    c = dict(case)
    Hq, Hkv = c["Hq"], c["Hkv"]
    if c["kind"] in ("prefill", "train"):
        B, T = c["B"], c["T"]
        c.update(q=normal(B, T, Hq, D), k=normal(B, T, Hkv, D), v=normal(B, T, Hkv, D),
                 g=normal(B, T, Hq, D, std=c["g_std"]))
        if c["kind"] == "train":
            c["dO"] = normal(B, T, Hq, D)
    else:
        N = c["N"]
        c.update(q=normal(N, Hq, D), k=normal(N, Hkv, D), v=normal(N, Hkv, D))
        if c["kind"] == "decode":
            c.update(g=normal(N, Hq, D), k_cache=normal(N, Hkv, W, D), v_cache=normal(N, Hkv, W, D),
                     k_sink=normal(N, Hkv, c["n_sink"], D), v_sink=normal(N, Hkv, c["n_sink"], D),
                     pos=torch.randint(c["lo"], c["hi"], (N,), generator=gen, device="cuda"))
        else:
            c.update(k_prefix=normal(1, Hkv, c["prefix"], D), v_prefix=normal(1, Hkv, c["prefix"], D),
                     k_cache=normal(N, Hkv, c["cap"], D), v_cache=normal(N, Hkv, c["cap"], D),
                     pos=c["prefix"] + torch.randint(0, c["cap"], (N,), generator=gen, device="cuda"))
    c["wq"] = 1.0 + 0.1 * torch.randn((D,), generator=gen, device="cuda")
    c["wk"] = 1.0 + 0.1 * torch.randn((D,), generator=gen, device="cuda")
    return c


# ---------------------------------------------------------------- one pass


def run(s):
    if own:
        return _run_own(s)
    with torch.no_grad():
        if s["kind"] == "prefill":
            return _sink_forward(s["q"].float(), s["k"].float(), s["v"].float(), s["g"].float(),
                                 s["wq"], s["wk"], s)[0].to(torch.bfloat16)
        if s["kind"] == "decode":
            return _sink_decode(s)
        if s["kind"] == "shared":
            return _shared_decode(s)
    return _sink_train(s)


def _run_own(s):
    import hybrid_sliding_window_gated_b200 as swa
    rope = dict(rot_dim=s["rot"], rope_base=s["base"], eps=EPS)
    if s["kind"] == "prefill":
        return swa.sink_fwd(s["q"], s["k"], s["v"], s["g"], s["wq"], s["wk"], s["n_sink"], **rope)
    if s["kind"] == "train":
        o, lse = swa.sink_fwd(s["q"], s["k"], s["v"], s["g"], s["wq"], s["wk"], s["n_sink"],
                              want_lse=True, **rope)
        grads = swa.sink_bwd(s["q"], s["k"], s["v"], s["g"], s["wq"], s["wk"], o, lse, s["dO"],
                             s["n_sink"], **rope)
        return [o] + [x.to(torch.bfloat16) for x in grads]
    if s["kind"] == "decode":
        o = swa.sink_decode_step(s["pos"], s["q"], s["k"], s["v"], s["g"], s["wq"], s["wk"],
                                 s["k_cache"], s["v_cache"], s["k_sink"], s["v_sink"], **rope)
        return [o, s["k_cache"], s["v_cache"], s["k_sink"], s["v_sink"]]
    o = swa.global_decode_shared(s["pos"], s["q"], s["k"], s["v"], s["wq"], s["wk"], s["k_prefix"],
                                 s["v_prefix"], s["prefix"], s["k_cache"], s["v_cache"], **rope)
    return [o, s["k_cache"], s["v_cache"]]


# -------------------------------------------------------------- plain forms


def _norm_rope(x, w, pos, rot, base):
    """RoPE_pos(x / rms(x) * w) for x [..., H, D] and pos of x's leading axes."""
    y = x * torch.rsqrt((x * x).mean(-1, keepdim=True) + EPS) * w
    if rot == 0:
        return y
    j = torch.arange(rot // 2, device=x.device, dtype=torch.float64)
    angle = pos.double()[..., None, None] * base ** (-2.0 * j / rot)
    cos, sin = angle.cos().float(), angle.sin().float()
    a, b, rest = y[..., :rot // 2], y[..., rot // 2:rot], y[..., rot:]
    return torch.cat([a * cos - b * sin, b * cos + a * sin, rest], -1)


def _sink_forward(q, k, v, g, wq, wk, s):
    """The sink attention of [B, T] tokens in blocks of W queries, each against
    its own and the previous block's keys and the sinks; returns o."""
    B, T, Hq = q.shape[:3]
    Hkv, S = k.shape[2], min(s["n_sink"], T)
    G, nb = Hq // Hkv, -(-T // W)
    pos = torch.arange(T, device=q.device)
    q = _norm_rope(q, wq, pos.expand(B, T), s["rot"], s["base"])
    k = _norm_rope(k, wk, pos.expand(B, T), s["rot"], s["base"])

    def blocks(x, H):  # [B, T, H, D] -> [B, H, nb, W, D]
        x = torch.nn.functional.pad(x, (0, 0, 0, 0, 0, nb * W - T))
        return x.reshape(B, nb, W, H, D).permute(0, 3, 1, 2, 4)

    def with_previous(x):  # [B, Hkv, nb, W, D] -> [B, Hkv, nb, 2 W, D]
        return torch.cat([torch.nn.functional.pad(x, (0, 0, 0, 0, 1, 0))[:, :, :-1], x], 3)

    qb = blocks(q, Hq).reshape(B, Hkv, G, nb, W, D).permute(0, 1, 3, 2, 4, 5).reshape(B, Hkv, nb, G * W, D)
    kb, vb = with_previous(blocks(k, Hkv)), with_previous(blocks(v, Hkv))
    ks = k[:, :S].permute(0, 2, 1, 3)  # [B, Hkv, S, D]
    vs = v[:, :S].permute(0, 2, 1, 3)
    band = torch.matmul(qb, kb.transpose(-1, -2))
    sink = torch.matmul(qb, ks.transpose(-1, -2)[:, :, None])
    blk = torch.arange(nb, device=q.device)[:, None, None]
    i = blk * W + torch.arange(W, device=q.device)[None, :, None]
    j = (blk - 1) * W + torch.arange(2 * W, device=q.device)[None, None, :]
    see = (j >= 0) & (j <= i) & (i - j < W)
    see = torch.cat([see, torch.arange(S, device=q.device)[None, None, :] <= i - W], -1)
    x = torch.cat([band, sink], -1).reshape(B, Hkv, nb, G, W, 2 * W + S) / math.sqrt(D)
    x = x.masked_fill(~see[:, None], -math.inf)
    m = x.detach().amax(-1, keepdim=True)
    p = (x - m).exp()
    p = (p / p.sum(-1, keepdim=True)).reshape(B, Hkv, nb, G * W, 2 * W + S)
    a = torch.matmul(p[..., :2 * W], vb) + torch.matmul(p[..., 2 * W:], vs[:, :, None])
    a = a.reshape(B, Hkv, nb, G, W, D).permute(0, 2, 4, 1, 3, 5).reshape(B, nb * W, Hq, D)[:, :T]
    return a * torch.sigmoid(g), see


def _sink_train(s):
    x = [s[n].float().requires_grad_() for n in ("q", "k", "v", "g")]
    x += [s[n].clone().requires_grad_() for n in ("wq", "wk")]
    with torch.enable_grad():
        o = _sink_forward(*x, s)[0]
    grads = torch.autograd.grad(o, x, s["dO"].float())
    # the gradients as they go into a training program's bf16 buckets
    return [o.detach().to(torch.bfloat16)] + [d.to(torch.bfloat16) for d in grads]


def _sink_decode(s):
    N, Hq, Hkv, S, pos = s["N"], s["Hq"], s["Hkv"], s["n_sink"], s["pos"]
    G, n = Hq // Hkv, torch.arange(N, device=pos.device)
    q = _norm_rope(s["q"].float(), s["wq"], pos, s["rot"], s["base"]).reshape(N, Hkv, G, D)
    k = _norm_rope(s["k"].float(), s["wk"], pos, s["rot"], s["base"]).to(torch.bfloat16)
    s["k_cache"][n, :, pos % W] = k
    s["v_cache"][n, :, pos % W] = s["v"]
    at = torch.arange(S, device=pos.device)
    early = (at == pos[:, None])[:, None, :, None]  # a token that is a sink itself
    s["k_sink"].copy_(torch.where(early, k[:, :, None], s["k_sink"]))
    s["v_sink"].copy_(torch.where(early, s["v"][:, :, None], s["v_sink"]))
    slot = torch.arange(W, device=pos.device)
    see = torch.cat([pos[:, None] - (pos[:, None] - slot) % W >= 0, at <= pos[:, None] - W], -1)
    kk = torch.cat([s["k_cache"], s["k_sink"]], 2).float()
    vv = torch.cat([s["v_cache"], s["v_sink"]], 2).float()
    x = torch.matmul(q, kk.transpose(-1, -2)) / math.sqrt(D)
    x = x.masked_fill(~see[:, None, None], -math.inf)
    p = (x - x.amax(-1, keepdim=True)).exp()
    a = torch.matmul(p / p.sum(-1, keepdim=True), vv).reshape(N, Hq, D)
    o = a * torch.sigmoid(s["g"].float())
    return [o.to(torch.bfloat16), s["k_cache"], s["v_cache"], s["k_sink"], s["v_sink"]]


def _shared_decode(s):
    N, Hq, Hkv, P, cap, pos = s["N"], s["Hq"], s["Hkv"], s["prefix"], s["cap"], s["pos"]
    G, n = Hq // Hkv, torch.arange(N, device=pos.device)
    q = _norm_rope(s["q"].float(), s["wq"], pos, s["rot"], s["base"]).reshape(N, Hkv, G, D)
    k = _norm_rope(s["k"].float(), s["wk"], pos, s["rot"], s["base"]).to(torch.bfloat16)
    s["k_cache"][n, :, pos - P] = k
    s["v_cache"][n, :, pos - P] = s["v"]
    # the prefix: all sequences' queries of a KV head against one K and V
    qp = q.permute(1, 0, 2, 3).reshape(Hkv, N * G, D)
    x0 = torch.matmul(qp, s["k_prefix"][0].float().transpose(-1, -2)) / math.sqrt(D)
    x0 = x0.reshape(Hkv, N, G, P).permute(1, 0, 2, 3)
    x1 = torch.matmul(q, s["k_cache"].float().transpose(-1, -2)) / math.sqrt(D)
    see = torch.arange(cap, device=pos.device) <= (pos - P)[:, None]
    x1 = x1.masked_fill(~see[:, None, None], -math.inf)
    m = torch.maximum(x0.amax(-1, keepdim=True), x1.amax(-1, keepdim=True))
    p0, p1 = (x0 - m).exp(), (x1 - m).exp()
    total = p0.sum(-1, keepdim=True) + p1.sum(-1, keepdim=True)
    a0 = torch.matmul(p0.permute(1, 0, 2, 3).reshape(Hkv, N * G, P), s["v_prefix"][0].float())
    a = a0.reshape(Hkv, N, G, D).permute(1, 0, 2, 3) + torch.matmul(p1, s["v_cache"].float())
    return [(a / total).reshape(N, Hq, D).to(torch.bfloat16), s["k_cache"], s["v_cache"]]


# -------------------------------------------------------------------- work


def _pairs(c):
    """Visible (query, key) pairs of one head over a prefill's tokens."""
    T, S = c["T"], c["n_sink"]
    n = min(T, W)
    in_window = n * (n + 1) // 2 + (T - n) * W
    # query i sees the sinks s <= min(S - 1, i - W) outside its window
    full = max(0, T - W - S)
    part = max(0, min(T - W, S))
    return c["B"] * (in_window + part * (part + 1) // 2 + full * S)


def work(c):
    Hq, Hkv = c["Hq"], c["Hkv"]
    row = 2 * D  # bytes of one bf16 row
    if c["kind"] == "prefill":
        t = c["B"] * c["T"]
        return dict(bytes=t * (3 * Hq + 2 * Hkv) * row, flops=4 * D * Hq * _pairs(c))
    if c["kind"] == "train":  # two products forward, five backward
        t = c["B"] * c["T"]
        return dict(bytes=t * (6 * Hq + 4 * Hkv) * row, flops=14 * D * Hq * _pairs(c))
    N = c["N"]
    if c["kind"] == "decode":
        ctx = W + c["n_sink"]
        return dict(bytes=N * row * (3 * Hq + Hkv * (2 * (ctx - 1) + 4)), flops=4 * D * Hq * N * ctx)
    ctx = c["prefix"] + (c["cap"] + 1) / 2  # the mean length of a drawn position
    return dict(bytes=row * Hkv * 2 * (c["prefix"] + N * (c["cap"] - 1) / 2) + N * row * (2 * Hq + 4 * Hkv),
                flops=4 * D * Hq * N * ctx)


# ------------------------------------------------------------ 64-bit values


def exact(case, seed):
    s = prepare(case, seed)
    with torch.no_grad():
        if s["kind"] == "decode" or s["kind"] == "shared":
            return _exact_decode(s)
        return _exact_tokens(s)


def _turn(y, pos, rot, base, back=False):
    """Rotates pair (j, j + rot/2) of y [rows, heads, D] by pos base^(-2j/rot), or back by it."""
    h = rot // 2
    z = y.clone()
    if h:
        f = torch.pow(torch.tensor(base, dtype=torch.float64, device=y.device),
                      -2.0 * torch.arange(h, dtype=torch.float64, device=y.device) / rot)
        c = torch.polar(torch.ones((), dtype=torch.float64, device=y.device),
                        pos.double()[:, None] * f * (-1.0 if back else 1.0))[:, None]
        t = torch.complex(y[..., :h].contiguous(), y[..., h:rot].contiguous()) * c
        z[..., :h], z[..., h:rot] = t.real, t.imag
    return z


def _unit(x):
    """x over its root mean square, and one over that."""
    r = 1.0 / torch.sqrt(x.pow(2).sum(-1, keepdim=True) / D + EPS)
    return x * r, r


def _exact_tokens(s):
    B, T, Hq, Hkv, S = s["B"], s["T"], s["Hq"], s["Hkv"], s["n_sink"]
    train, G, dev = s["kind"] == "train", Hq // Hkv, s["q"].device
    wq, wk, step = s["wq"].double(), s["wk"].double(), 1024
    out = torch.empty(s["q"].shape, dtype=torch.float64 if train else torch.float32, device=dev)
    if train:
        dq, dg = torch.zeros_like(out), torch.zeros_like(out)
        dk = torch.zeros(s["k"].shape, dtype=torch.float64, device=dev)
        dv, dwq, dwk = torch.zeros_like(dk), torch.zeros_like(wq), torch.zeros_like(wk)
    near = torch.arange(W - 1, -1, -1, device=dev)
    first = torch.arange(S, device=dev)
    where = torch.arange(T, device=dev)
    for b in range(B):
        for h in range(Hkv):
            heads = slice(h * G, h * G + G)
            ku, kr = _unit(s["k"][b, :, h].double())
            kk = _turn((ku * wk)[:, None], where, s["rot"], s["base"])[:, 0]
            vv = s["v"][b, :, h].double()
            dkk = torch.zeros_like(kk)
            for i0 in range(0, T, step):
                i = where[i0:i0 + step]
                # the keys of each query: its window, then the sinks outside it
                idx = torch.cat([i[:, None] - near, first.expand(len(i), S)], 1)
                ok = torch.cat([i[:, None] >= near, first <= i[:, None] - W], 1)
                idx = torch.where(ok, idx, 0)
                qu, qr = _unit(s["q"][b, i, heads].double())
                qq = _turn(qu * wq, i, s["rot"], s["base"])
                ki, vi = kk[idx], vv[idx]
                x = torch.einsum("rgd,rkd->rgk", qq, ki) * D ** -0.5
                p = torch.softmax(torch.where(ok[:, None], x, -math.inf), -1)
                a = torch.einsum("rgk,rkd->rgd", p, vi)
                gate = 1.0 / (1.0 + torch.exp(-s["g"][b, i, heads].double()))
                out[b, i, heads] = (a * gate).to(out.dtype)
                if not train:
                    continue
                do = s["dO"][b, i, heads].double()
                da = do * gate
                dg[b, i, heads] = do * a * gate * (1.0 - gate)
                dx = p * (torch.einsum("rgd,rkd->rgk", da, vi) - (da * a).sum(-1, keepdim=True)) * D ** -0.5
                dqq = _turn(torch.einsum("rgk,rkd->rgd", dx, ki), i, s["rot"], s["base"], back=True)
                dwq += (dqq * qu).sum((0, 1))
                du = dqq * wq
                dq[b, i, heads] = qr * (du - qu * (du * qu).mean(-1, keepdim=True))
                flat = idx.reshape(-1)
                dkk.index_add_(0, flat, torch.einsum("rgk,rgd->rkd", dx, qq).reshape(-1, D))
                dv[b, :, h].index_add_(0, flat, torch.einsum("rgk,rgd->rkd", p, da).reshape(-1, D))
            if train:
                dkk = _turn(dkk[:, None], where, s["rot"], s["base"], back=True)[:, 0]
                dwk += (dkk * ku).sum(0)
                du = dkk * wk
                dk[b, :, h] = kr * (du - ku * (du * ku).mean(-1, keepdim=True))
    return [out, dq, dk, dv, dg, dwq, dwk] if train else out


def _exact_decode(s):
    N, Hq, Hkv, pos = s["N"], s["Hq"], s["Hkv"], s["pos"]
    G, sink = Hq // Hkv, s["kind"] == "decode"
    q = _turn(_unit(s["q"].double())[0] * s["wq"].double(), pos, s["rot"], s["base"])
    k = _turn(_unit(s["k"].double())[0] * s["wk"].double(), pos, s["rot"], s["base"])
    k = k.to(torch.bfloat16)  # the cache holds bf16
    o = torch.empty(s["q"].shape, dtype=torch.float64, device=pos.device)
    for n, p in enumerate(pos.tolist()):
        slot = p % W if sink else p - s["prefix"]
        s["k_cache"][n, :, slot], s["v_cache"][n, :, slot] = k[n], s["v"][n]
        if sink:
            if p < s["n_sink"]:
                s["k_sink"][n, :, p], s["v_sink"][n, :, p] = k[n], s["v"][n]
            # the context in the order of the positions: sinks, then the window
            early = max(0, min(s["n_sink"], p - W + 1))
            held = [t % W for t in range(max(0, p - W + 1), p + 1)]
            kk = torch.cat([s["k_sink"][n, :, :early], s["k_cache"][n][:, held]], 1).double()
            vv = torch.cat([s["v_sink"][n, :, :early], s["v_cache"][n][:, held]], 1).double()
            x = torch.einsum("hgd,hkd->hgk", q[n].reshape(Hkv, G, D), kk) * D ** -0.5
            a = torch.einsum("hgk,hkd->hgd", torch.softmax(x, -1), vv).reshape(Hq, D)
            o[n] = a / (1.0 + torch.exp(-s["g"][n].double()))
        else:
            for h in range(Hkv):
                kk = torch.cat([s["k_prefix"][0, h], s["k_cache"][n, h, :slot + 1]]).double()
                vv = torch.cat([s["v_prefix"][0, h], s["v_cache"][n, h, :slot + 1]]).double()
                x = torch.einsum("gd,kd->gk", q[n, h * G:h * G + G], kk) * D ** -0.5
                o[n, h * G:h * G + G] = torch.softmax(x, -1) @ vv
    caches = [s["k_cache"], s["v_cache"]] + ([s["k_sink"], s["v_sink"]] if sink else [])
    return [o] + caches
