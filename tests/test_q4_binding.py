"""Host-only checks of the binding of the rotary, paged-append and 4-bit KV calls
(no GPU): what reaches the library is what the caller passed."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")


def _dsb():
    from session_decode_step_dsb_gb300 import dsb
    return dsb


BATCH = dict(block_table=[[0, 1], [2, 3]], n_blocks=[2, 2], window=[0, 0], new_tokens=[1, 2], seq_lens=[130, 2])
BAD = [np.array([(1 << 32) + 1, 2]), np.array([1, -(1 << 32) + 2]), np.array([1, 1 << 31], np.uint32), [1, (1 << 31)],
       np.array([1.5, 2.0]), np.array([1.0, np.nan]), np.array([1.0, np.inf]), ["1", "2"]]


@pytest.mark.parametrize("bad", BAD)
@pytest.mark.parametrize("name", list(BATCH))
def test_batches_take_only_what_int32_holds(name, bad):
    d = _dsb()
    value = [bad, bad] if name == "block_table" else bad
    with pytest.raises(ValueError, match=name):
        d.PagedBatch(**{**BATCH, name: value})


@pytest.mark.parametrize("bad", BAD)
def test_positions_and_spans_take_only_what_int32_holds(bad):
    d = _dsb()
    with pytest.raises(ValueError, match="pos must hold"):
        d.rope_rotary(torch.zeros((2, 4, 64)), None, bad, d.Rotary(), None)
    kv = d.KVQ4Pages(1 << 20, 8, 2, 64)
    kv._tensors = (torch.zeros((8, 2, 128 * 72), dtype=torch.uint8),)
    batch = d.PagedBatch(**BATCH)
    with pytest.raises(ValueError, match="first must hold"):
        d.kv_gather_q4(kv, batch, bad, [1, 1], d.DSB_F16, None)
    with pytest.raises(ValueError, match="count must hold"):
        d.kv_gather_q4(kv, batch, [0, 0], bad, d.DSB_F16, None)


@pytest.mark.parametrize("kind", [np.int8, np.uint8, np.int16, np.int64, np.uint64, np.float32, np.float64, bool, list])
def test_whole_numbers_of_any_type_arrive(kind):
    """And as a copy: the batch is not the caller's array."""
    d = _dsb()
    arrays = {k: np.array(v) for k, v in BATCH.items()}
    arrays["new_tokens"] = [1, 0] if kind is list else np.array([1, 0]).astype(kind)
    b = d.PagedBatch(**arrays)
    assert [b.c.new_tokens[i] for i in range(2)] == [1, 0] and [b.c.seq_lens[i] for i in range(2)] == [130, 2]
    own = np.array([1, 2], np.int32)
    b = d.PagedBatch(**{**BATCH, "new_tokens": own})
    own[:] = 9
    assert [b.c.new_tokens[i] for i in range(2)] == [1, 2]
    arr, at = d._host_i32(own, 2, "x")
    assert arr is own and at == own.ctypes.data
    assert d._host_i32(np.array([3, 4, 5, 6])[::2], 2, "x")[0].tolist() == [3, 5]


def test_what_a_call_makes_belongs_to_its_stream(monkeypatch):
    """The handle 0 is the default stream's; other handles are wrapped, streams
    taken as they are."""
    import contextlib
    d, entered = _dsb(), []

    class Stream:
        def __init__(self, name):
            self.name = name

    @contextlib.contextmanager
    def on(stream):
        entered.append(stream.name)
        yield

    monkeypatch.setattr(torch.cuda, "Stream", Stream)
    monkeypatch.setattr(torch.cuda, "ExternalStream", lambda handle, device: Stream(("handle", handle, device)))
    monkeypatch.setattr(torch.cuda, "default_stream", lambda device: Stream(("default", device)))
    monkeypatch.setattr(torch.cuda, "stream", on)
    for stream in (0, 77, Stream("given"), None):
        assert d._empty_on(stream, (2, 3), torch.float32, "cpu").shape == (2, 3)
    assert entered == [("default", "cpu"), ("handle", 77, "cpu"), "given"]
