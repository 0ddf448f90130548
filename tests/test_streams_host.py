"""What the bindings allocate for a call on another stream than the current one, on the CPU.

The library is a stub that takes the calls' pointers; every tensor made inside a
call has to be handed to the allocator's bookkeeping for that stream, since its
memory may still be in use, or be used again, on the current one."""
import ctypes

import pytest

from bit_quantized_lm_amd import _binding as B

torch = pytest.importorskip("torch")


class Stub:
    """A library whose functions remember the pointers that they get."""

    def __init__(self):
        self.pointers = set()

    def __getattr__(self, name):
        def call(*args):
            for a in args:
                value = a.value if isinstance(a, ctypes.c_void_p) else a if isinstance(a, int) else None
                if value and value > 1 << 20:
                    self.pointers.add(value)
            return 0
        return call


@pytest.fixture
def run(monkeypatch):
    """run(f): calls f(stream); the addresses that the library got and the tensors kept for the stream."""
    stub, kept = Stub(), []
    monkeypatch.setattr(B, "load_library", lambda: stub)
    monkeypatch.setattr(B, "draft_head_workspace_bytes", lambda M, K: 4096)
    monkeypatch.setattr(B, "_stream", lambda s: None)
    monkeypatch.setattr(B, "_keep_for", lambda made, stream: kept.extend(made) if stream is not None else None)

    def go(f, *given):
        f("side")
        known = {t.data_ptr() for t in kept} | {t.data_ptr() for t in given}
        assert stub.pointers <= known, "a tensor that was made here is not kept for the stream"
        assert kept and stub.pointers & {t.data_ptr() for t in kept}
        return kept
    return go


M, K, N, R = 3, 512, 200, 16


def tensors():
    ids, vals = torch.zeros((M, R), dtype=torch.int32), torch.zeros((M, R))
    cand = torch.zeros((M, 32)), torch.zeros((M, 32), dtype=torch.int32)
    return {"x": torch.zeros((M, K), dtype=torch.bfloat16), "tiled": torch.zeros(4096, dtype=torch.uint8), "pairs": torch.zeros(4096, dtype=torch.int32),
            "w": torch.zeros((N, K), dtype=torch.int16), "ids": ids, "vals": vals, "cv": cand[0], "ci": cand[1], "scale": torch.zeros(N)}


CALLS = {
    "coarse": lambda t, s: B.draft_head_coarse(t["x"], t["tiled"], t["pairs"], N, stream=s),
    "rerank": lambda t, s: B.draft_head_rerank(t["x"], t["w"], t["cv"], t["ci"], R, stream=s),
    "rerank_e4m3": lambda t, s: B.draft_head_rerank_e4m3(t["x"], t["w"], t["scale"], t["cv"], t["ci"], R, stream=s),
    "rerank_nvfp4": lambda t, s: B.draft_head_rerank_nvfp4(t["x"], t["w"], t["w"], t["scale"], t["cv"], t["ci"], R, stream=s),
    "logits_row": lambda t, s: B.draft_head_logits_row(t["ids"], t["vals"], N, stream=s),
    "stream_read": lambda t, s: B.draft_head_stream_read(t["tiled"], stream=s),
    "argmax": lambda t, s: B.draft_head_argmax(t["ids"], t["vals"], stream=s),
    "forward": lambda t, s: B.draft_head_forward(t["x"], t["tiled"], t["pairs"], t["w"], N, stream=s),
    "forward_row": lambda t, s: B.draft_head_forward_row(t["x"], t["tiled"], t["pairs"], t["w"], N, stream=s),
    "forward_noalloc": lambda t, s: B.draft_head_forward_noalloc(t["x"], t["tiled"], t["pairs"], t["w"], N, stream=s),
    "staged row": lambda t, s: B.DraftHead(t["tiled"], t["pairs"], t["w"], N, K).logits_row_staged(t["x"], stream=s),
    "staged": lambda t, s: B.DraftHead(t["tiled"], t["pairs"], t["w"], N, K).staged(t["x"], stream=s),
}


@pytest.mark.parametrize("name", CALLS)
def test_what_a_call_makes_is_kept_for_its_stream(run, name):
    t = tensors()
    run(lambda s: CALLS[name](t, s), *t.values())


def test_what_the_caller_gives_is_the_callers(run):
    t = tensors()
    out = B.forward_buffers(M, N, 8, 32, "cpu")
    mine = [*out.values(), torch.zeros((M, N), dtype=torch.int16), torch.zeros(4096, dtype=torch.uint8)]
    with pytest.raises(AssertionError):      # nothing is made, so nothing is kept
        run(lambda s: B.draft_head_forward_row(t["x"], t["tiled"], t["pairs"], t["w"], N, out=out, row=mine[-2], workspace=mine[-1], stream=s),
            *t.values(), *mine)


def test_the_streams_order():
    """keep_for: nothing for the current stream, one wait and a record a tensor for another."""
    log = []

    class Stream:
        def __init__(self, handle):
            self.cuda_stream = handle

        def wait_stream(self, other):
            log.append(("wait", self.cuda_stream, other.cuda_stream))

    class Tensor:
        device = "cuda:0"

        def record_stream(self, s):
            log.append(("record", s.cuda_stream))

    here = Stream(5)
    with pytest.MonkeyPatch.context() as m:
        m.setattr(torch.cuda, "current_stream", lambda dev=None: here)
        m.setattr(torch.cuda, "default_stream", lambda dev=None: Stream(0))
        m.setattr(torch.cuda, "ExternalStream", lambda handle, device=None: Stream(handle))
        two = [Tensor(), Tensor()]
        B._keep_for(two, None)
        B._keep_for([], Stream(7))
        B._keep_for(two, Stream(5))
        B._keep_for(two, 5)
        assert not log
        B._keep_for(two, Stream(7))
        assert log == [("wait", 7, 5), ("record", 7), ("record", 7)]
        del log[:]
        B._keep_for(two[:1], 0)
        assert log == [("wait", 0, 5), ("record", 0)]
