"""The two buffers of a Workspace, without a GPU."""
import gc
import weakref

import torch

import int8_w8a8_quantized_smoothed_b200 as w8


def test_calls_that_leave_any_contents_never_get_the_zeroed_buffer():
    """The GEMMs take nonzero flag words for partial results that are ready, so what the gradient
    calls write has to go elsewhere, in either order and when the buffers grow."""
    ws = w8.Workspace("cpu")
    like = torch.empty(0)
    zeroed, _ = ws.get(8192)
    for nbytes in (4096, 1 << 21, 64):
        ptr, size, buf = w8._scratch(ws, nbytes, like, -1)
        assert size >= nbytes and ptr == buf.data_ptr()
        buf.fill_(0xFF)
        assert ws.get(8192)[0].data_ptr() == zeroed.data_ptr()
        assert not zeroed.any()
    grown, _ = ws.get(1 << 22)
    assert not grown.any() and w8._scratch(ws, 64, like, -1)[2].data_ptr() != grown.data_ptr()


def test_nothing_is_handed_out_for_nothing():
    ws = w8.Workspace("cpu")
    assert w8._scratch(ws, 0, torch.empty(0), -1) == (None, 0, None)
    assert ws.get(0) == (None, 0) and ws.buf is None and not ws.scratch_bufs


def test_an_outgrown_buffer_stays():
    """A graph captured with it writes to it on every replay."""
    ws = w8.Workspace("cpu")
    first = weakref.ref(ws.scratch(1000))
    assert ws.scratch(1001).numel() == 2000
    assert ws.scratch(5000).numel() == 5000
    gc.collect()
    assert first() is not None and first().numel() == 1000


def test_a_callers_tensor_and_a_new_one():
    mine = torch.empty(128, dtype=torch.float32)
    ptr, size, _ = w8._scratch(mine, 512, torch.empty(0), -1)
    assert ptr == mine.data_ptr() and size == 512
    a, b = (w8._scratch(None, 512, torch.empty(0), -1)[2] for _ in range(2))
    assert a.numel() == 512 and a.data_ptr() != b.data_ptr()
