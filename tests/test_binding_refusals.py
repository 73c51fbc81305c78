"""CPU: what the binding refuses before the library sees it."""
import types

import pytest
import torch

import hybrid_sliding_window_gated_b200 as swa
from hybrid_sliding_window_gated_b200 import build as swa_build


class Elsewhere:
    """As much of a CUDA tensor as the checks ahead of a launch look at."""

    def __init__(self, shape, dtype, index=0):
        self.shape, self.dtype, self.device = torch.Size(shape), dtype, torch.device("cuda", index)
        self.is_cuda = True

    def numel(self):
        return self.shape.numel()

    def is_contiguous(self):
        return True

    def get_device(self):
        return self.device.index

    def dim(self):
        return len(self.shape)

    def data_ptr(self):
        return 0x1000


def inputs():
    bf, f32 = torch.bfloat16, torch.float32
    t = lambda *s, dtype=bf: Elsewhere(s, dtype)
    q, k, w = t(1, 8, 2, 128), t(1, 8, 1, 128), t(128, dtype=f32)
    one, new = t(1, 2, 128), t(1, 1, 128)
    pos = t(1, dtype=torch.int64)
    lse, ring = t(1, 2, 8, dtype=f32), t(1, 1, 128, 128)
    big = t(1 << 30, dtype=torch.uint8)
    grads = (q, k, k, q, w, w)
    return types.SimpleNamespace(**locals())


CALLS = {
    "fwd": lambda x: swa.fwd(x.q, x.k, x.k, x.q, x.w, x.w, out=x.q),
    "fwd_halo": lambda x: swa.fwd_halo(x.q, x.k, x.k, x.q, x.w, x.w, None, None, 0, out=x.q),
    "bwd": lambda x: swa.bwd(x.q, x.k, x.k, x.q, x.w, x.w, x.lse, x.q, workspace=x.big,
                             grads=x.grads),
    "bwd_noalloc": lambda x: swa.bwd_noalloc(x.q, x.k, x.k, x.q, x.w, x.w, x.lse, x.q,
                                             grads=x.grads),
    "decode_step": lambda x: swa.decode_step(x.pos, x.one, x.new, x.new, x.one, x.w, x.w, x.ring,
                                             x.ring, out=x.one),
    "prefill_to_ring": lambda x: swa.prefill_to_ring(x.k, x.k, x.w, x.ring, x.ring, Hq=2),
    "global_fwd": lambda x: swa.global_fwd(x.q, x.k, x.k, x.w, x.w, x.ring, x.ring, out=x.q),
    "global_decode_step": lambda x: swa.global_decode_step(x.pos, x.one, x.new, x.new, x.w, x.w,
                                                           x.ring, x.ring, out=x.one,
                                                           workspace=x.big),
    "sink_fwd": lambda x: swa.sink_fwd(x.q, x.k, x.k, x.q, x.w, x.w, 4, out=x.q),
    "sink_bwd": lambda x: swa.sink_bwd(x.q, x.k, x.k, x.q, x.w, x.w, x.q, x.lse, x.q, 4,
                                       workspace=x.big, grads=x.grads),
    "sink_decode_step": lambda x: swa.sink_decode_step(x.pos, x.one, x.new, x.new, x.one, x.w, x.w,
                                                       x.ring, x.ring, x.k, x.k, out=x.one),
    "global_decode_shared": lambda x: swa.global_decode_shared(
        x.pos, x.one, x.new, x.new, x.w, x.w, x.ring, x.ring, 16, x.ring, x.ring, out=x.one,
        workspace=x.big),
}


@pytest.mark.parametrize("name", CALLS)
def test_tensors_on_another_device_than_the_current_one(name, monkeypatch):
    """The library launches on the current device: the pointers are another's there."""
    swa_build.build()
    monkeypatch.setattr(swa, "_current_device", lambda: 1)
    launched = []
    for f in ("fwd", "fwd_halo", "bwd", "bwd_noalloc", "decode_step", "prefill_to_ring",
              "global_fwd", "global_decode_step", "sink_fwd", "sink_bwd", "sink_decode_step",
              "global_decode_shared"):
        monkeypatch.setattr(swa.lib(), "swa_" + f, lambda *a: launched.append(a) or 0)
    monkeypatch.setattr(swa, "_stream", lambda s: 0)
    with pytest.raises(ValueError, match="current device is cuda:1"):
        CALLS[name](inputs())
    assert not launched
    monkeypatch.setattr(swa, "_current_device", lambda: 0)
    CALLS[name](inputs())
    assert len(launched) == 1


def launches(monkeypatch, *names):
    swa_build.build()
    monkeypatch.setattr(swa, "_current_device", lambda: 0)
    monkeypatch.setattr(swa, "_stream", lambda s: 0)
    seen = []
    for f in names:
        monkeypatch.setattr(swa.lib(), "swa_" + f, lambda *a: seen.append(a) or 0)
    return seen


def test_decode_step_without_sink_caches(monkeypatch):
    """No caches, as in the C call, are no sinks; one without the other is a mistake."""
    seen = launches(monkeypatch, "sink_decode_step")
    x = inputs()
    call = lambda ks, vs: swa.sink_decode_step(x.pos, x.one, x.new, x.new, x.one, x.w, x.w, x.ring,
                                               x.ring, ks, vs, out=x.one)
    call(None, None)
    assert seen[0][1] == 0 and seen[0][11] is None and seen[0][12] is None
    c = types.SimpleNamespace(**{n: torch.zeros(t.shape, dtype=t.dtype) for n, t in vars(x).items()
                                 if n in ("pos", "one", "new", "w", "ring", "k")})
    for pair in ((c.k, None), (None, c.k)):
        with pytest.raises(TypeError, match="_sink must be a torch.Tensor"):
            swa.sink_decode_step(c.pos, c.one, c.new, c.new, c.one, c.w, c.w, c.ring, c.ring, *pair)


def test_caches_of_unlike_sizes(monkeypatch):
    """K and V caches of one call share their capacity: the larger one is no valid V cache."""
    seen = launches(monkeypatch, "sink_decode_step", "prefill_to_sinks", "global_decode_shared")
    x = inputs()
    bf = torch.bfloat16
    sink = [Elsewhere((1, 1, n, 128), bf) for n in (4, 5)]
    long, wide = Elsewhere((1, 1, 256, 128), bf), Elsewhere((1, 2, 128, 128), bf)

    def decode(vc, vs):
        swa.sink_decode_step(x.pos, x.one, x.new, x.new, x.one, x.w, x.w, x.ring, vc, sink[0], vs,
                             out=x.one)

    def shared(kp, vp, vc):
        swa.global_decode_shared(x.pos, x.one, x.new, x.new, x.w, x.w, kp, vp, 16, x.ring, vc,
                                 out=x.one, workspace=x.big)

    for match, call in [
        ("v_cache", lambda: decode(long, sink[0])),
        ("v_sink", lambda: decode(x.ring, sink[1])),
        ("v_sink", lambda: swa.prefill_to_sinks(x.k, x.k, x.w, *sink, Hq=2)),
        ("v_prefix", lambda: shared(x.ring, long, x.ring)),
        ("v_cache", lambda: shared(x.ring, x.ring, long)),
        ("2 heads", lambda: shared(wide, wide, x.ring)),
    ]:
        with pytest.raises(ValueError, match=match):
            call()
    assert not seen
    decode(x.ring, sink[0])
    swa.prefill_to_sinks(x.k, x.k, x.w, sink[0], sink[0], Hq=2)
    shared(x.ring, x.ring, x.ring)
    assert len(seen) == 3
