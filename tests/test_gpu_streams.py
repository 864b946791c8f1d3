"""Calls on a given stream: what they allocate belongs to that stream, so that it never lies on memory
that kernels of the current stream still use. Calls that wait for the GPU's queue: other threads run."""
import threading
import time

import pytest
import torch

from paged_kv_cache_147_gb300 import pkv

pytestmark = pytest.mark.gpu
DEV = "cuda"


def _pool_stream(t):
    """The stream whose pool of the caching allocator holds t."""
    at = t.data_ptr()
    for seg in torch.cuda.memory_snapshot():
        if seg["address"] <= at < seg["address"] + seg["total_size"]:
            return seg["stream"]
    raise AssertionError("not the allocator's")


def _calls(stream):
    i32 = dict(dtype=torch.int32, device=DEV)
    f16 = dict(dtype=torch.float16, device=DEV)
    table, lens, new = torch.full((2, 4), -1, **i32), torch.zeros(2, **i32), torch.ones(2, **i32)
    free, count = torch.arange(8, **i32), torch.full((1,), 8, **i32)
    q, k, w = torch.randn(3, 4, 128, **f16), torch.randn(3, 2, 128, **f16), torch.ones(128, **f16)
    pos, cs = torch.zeros(3, dtype=torch.int64, device=DEV), pkv.rope_table(4).to(DEV)
    seq, full = torch.zeros(3, **i32), torch.zeros(2, 4, **i32)
    logits, draft = torch.randn(2, 3, 50, device=DEV), torch.randn(2, 2, 50, device=DEV)
    u, drafts = torch.rand(2, 2, device=DEV), torch.zeros(2, 2, **i32)
    torch.cuda.synchronize()
    yield "norm", pkv.qk_norm_rope(q, k, w, w, 1e-6, pos, cs, stream=stream)
    yield "extend", pkv.extend_tables(table, lens, new, 16, free, count, 5, stream=stream)
    yield "slots", (pkv.slot_mapping(seq, pos, full, 16, stream=stream),)
    yield "ring slots", (pkv.ring_slot_mapping(seq, pos, full, 4, 32, 16, stream=stream),)
    yield "verify", pkv.spec_verify(logits, draft, drafts, u, u[:, 0].contiguous(), stream=stream)
    yield "workspace", (pkv.make_workspace(2, 1, 4, 2, stream=stream),)
    torch.cuda.synchronize()


def test_outputs_of_a_call_on_a_given_stream_belong_to_it():
    side = torch.cuda.Stream()
    for stream in (side, torch.cuda.ExternalStream(side.cuda_stream)):
        for what, outs in _calls(stream):
            assert [_pool_stream(t) for t in outs] == [side.cuda_stream] * len(outs), what
    main = torch.cuda.current_stream()
    for what, outs in _calls(None):
        assert [_pool_stream(t) for t in outs] == [main.cuda_stream] * len(outs), what
    for what, outs in _calls(main):     # the default stream, named
        assert [_pool_stream(t) for t in outs] == [main.cuda_stream] * len(outs), what
    assert torch.cuda.current_stream() == main
    assert pkv.device_error(clear=True) == 0


def test_a_stream_may_be_any_object_with_a_handle():
    class Handle:
        def __init__(self, value):
            self.cuda_stream = value

    side = torch.cuda.Stream()
    # a stream of another library's making; the default stream by both of its handles
    for handle, want in ((side.cuda_stream, side.cuda_stream), (0, 0), (1, 0)):
        for what, outs in _calls(Handle(handle)):
            assert [_pool_stream(t) for t in outs] == [want] * len(outs), (what, handle)
    assert pkv.device_error(clear=True) == 0


def test_a_call_inside_a_stream_context_gives_outputs_of_that_stream():
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        for what, outs in _calls(None):
            assert [_pool_stream(t) for t in outs] == [side.cuda_stream] * len(outs), what
    assert pkv.device_error(clear=True) == 0


def test_a_call_that_waits_for_the_queue_lets_other_threads_run():
    i32 = dict(dtype=torch.int32, device=DEV)
    table, lens, keep = torch.full((2, 4), -1, **i32), torch.zeros(2, **i32), torch.zeros(2, **i32)
    free, count = torch.arange(8, **i32), torch.full((1,), 8, **i32)
    gaps, done = [0.0], threading.Event()

    def watch():
        last = time.monotonic()
        while not done.is_set():
            time.sleep(0.002)
            now = time.monotonic()
            gaps.append(now - last)
            last = now

    pkv.truncate_tables(table, lens, keep, 16, free, count)
    torch.cuda.synchronize()
    thread = threading.Thread(target=watch)
    thread.start()
    waited = 0.0
    torch.cuda._sleep(2_000_000_000)      # about a second: the calls behind it fill the queue
    for _ in range(4000):
        before = time.monotonic()
        pkv.truncate_tables(table, lens, keep, 16, free, count)
        waited = max(waited, time.monotonic() - before)
    done.set()
    thread.join()
    torch.cuda.synchronize()
    assert waited > 0.3, "no call had to wait"
    assert max(gaps) < waited / 2, (max(gaps), waited)
