"""What a call allocates belongs to the stream it runs on: with ``stream=`` every output and workspace comes from that
stream's pool (a block of the current stream's could still be in use there, and would go back to it while the kernels
run), and outputs are marked as read on the current stream.  No GPU: the allocations are watched up to the refusal of
host tensors."""
import contextlib
from functools import partial

import pytest
import torch


@pytest.fixture(scope="module")
def bi():
    from invariant_fixed_order_gb300 import build
    build.build()
    from invariant_fixed_order_gb300 import bi as b
    return b


class Watched(torch.Tensor):
    """A host tensor that notes record_stream."""
    marked = None

    def record_stream(self, stream):
        self.marked = stream


class Logits(Watched):
    """Passes for a device tensor where is_cuda is asked (token_logprobs asks it before it allocates)."""
    is_cuda = True


def host(*shape, dt=torch.bfloat16):
    return torch.zeros(*shape, dtype=dt).as_subclass(Watched)


I32, F32 = torch.int32, torch.float32


def calls(bi):
    q, cache, table = host(2, 8, 64), host(5, 2, 16, 64), host(2, 4, dt=I32)
    logits = host(2, 100, dt=F32)
    one = host(2, dt=I32)
    return {
        "rmsnorm": (1, 0, partial(bi.rmsnorm, host(2, 128), host(128))),
        "gemm": (1, 0, partial(bi.gemm, host(4, 128), host(128, 128))),
        "pack_gate_up": (1, 0, partial(bi.pack_gate_up, host(32, 128), host(32, 128))),
        "decode_attention": (1, 1, partial(bi.decode_attention, q, cache, cache, table, one, 64)),
        "decode_attention_noalloc": (1, 0, partial(bi.decode_attention_noalloc, q, cache, cache, table, one, 64)),
        "prefill_attention": (1, 0, partial(bi.prefill_attention, q, host(3, dt=I32), one, cache, cache, table)),
        "argmax": (1, 0, partial(bi.argmax, logits)),
        "log_softmax": (1, 1, partial(bi.log_softmax, logits)),
        "sample": (1, 1, partial(bi.sample, logits, one, one, host(2, dt=F32))),
        "embed": (1, 0, partial(bi.embed, host(9, 64), one)),
        "build_slots": (4, 0, partial(bi.build_slots, one, one, table, one, host(1, dt=I32), 4, 9)),
        "tree_attention": (1, 1, partial(bi.tree_attention, q, host(3, dt=I32), one, host(2, 1, dt=I32), cache, cache,
                                          table, 8)),
        "token_logprobs": (4, 1, partial(bi.token_logprobs, logits.as_subclass(Logits), host(2, 1, dt=I32), top_k=3)),
    }


NAMES = ["rmsnorm", "gemm", "pack_gate_up", "decode_attention", "decode_attention_noalloc", "prefill_attention", "argmax",
         "log_softmax", "sample", "embed", "build_slots", "tree_attention", "token_logprobs"]


@pytest.mark.parametrize("name", NAMES)
def test_a_calls_memory_is_its_streams(bi, monkeypatch, name):
    results, scratch, call = calls(bi)[name]
    within, made = [], []

    @contextlib.contextmanager
    def on(stream):
        within.append(stream)
        yield
        within.pop()

    def watch(make):
        def made_on(*shape, **kw):
            t = make(*shape, **kw).as_subclass(Watched)
            made.append((t, within[-1] if within else None))
            return t
        return made_on

    for f in ("empty", "empty_like", "full", "zeros"):
        monkeypatch.setattr(torch, f, watch(getattr(torch, f)))
    monkeypatch.setattr(torch.cuda, "stream", on)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda device=None: "current")
    with pytest.raises(ValueError, match="expected a CUDA tensor"):
        call(stream="launch")
    assert len(made) == results + scratch
    assert all(stream == "launch" for _, stream in made)
    assert sum(t.marked == "current" for t, _ in made) == results
    made.clear()
    with pytest.raises(ValueError, match="expected a CUDA tensor"):
        call()
    assert len(made) == results + scratch and all(stream is None for _, stream in made)
