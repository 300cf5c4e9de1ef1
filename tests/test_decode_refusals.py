"""Refusals of the decode operators' torch layer on the CPU: arguments whose
sizes say more than their memory holds. (Tensors stay on the host; the device
check is put aside, and every call is refused before any entry point.)"""

import pytest
import torch

from quantized_weight_skinny_amd import decode_api as qd

CPU = torch.device("cpu")


@pytest.fixture
def on_host(monkeypatch):
    monkeypatch.setattr(qd, "_on_device", lambda *a: None)


def test_a_workspace_must_be_contiguous(on_host):
    """An expanded tensor has elements that its storage does not, and between
    those of a strided one lie somebody else's."""
    for ws in (torch.empty(1, dtype=torch.uint8).expand(4096), torch.empty(8192, dtype=torch.uint8)[::2],
               torch.empty((64, 64), dtype=torch.uint8)[:, :32], torch.empty((64, 64), dtype=torch.float32).t()):
        with pytest.raises(ValueError, match="contiguous"):
            qd._workspace(1024, ws, CPU)
    ws = torch.empty((16, 64), dtype=torch.float32)
    assert qd._workspace(4096, ws, CPU) == (ws, ws.data_ptr(), 4096)
    assert qd._workspace(0, None, CPU) == (None, None, 0)
    assert qd._workspace(4097, ws, CPU)[0] is not ws       # too small: a new one


def test_attention_takes_no_longer_bound_than_the_table_holds(on_host):
    """A slice of a wider table: its rows lie further apart than they are long,
    and a bound beyond their length would look up pages past them."""
    cache = qd.KV4Cache(4, 16, 2, 64, device="cpu")
    q, lengths = torch.zeros((2, 4, 64), dtype=torch.float16), torch.zeros(2, dtype=torch.int32)
    wide = torch.zeros((2, 50), dtype=torch.int32)
    for table in (wide[:, :3], wide[:, 47:], wide[:, 3:6].contiguous()):
        for bound in (49, 800):
            with pytest.raises(ValueError, match="max_kv_len"):
                qd.kv4_attention(q, cache, table, lengths, max_kv_len=bound)
    with pytest.raises(ValueError, match="max_kv_len"):
        qd.kv4_attention(q, cache, wide[:, :0], lengths, max_kv_len=1)


def test_a_caches_fields_do_not_change():
    """Its descriptors are built once a layer; a field replaced afterwards would
    leave the calls at the old buffer (sizes, scales)."""
    cache = qd.KV4Cache(4, 16, 2, 64, layers=2, device="cpu")
    for name, value in (("data", cache.data.clone()), ("k_scale", (1.0, 1.0)), ("v_scale", (1.0, 1.0)), ("pages", 3),
                        ("page_size", 32), ("kv_heads", 1), ("head_dim", 128), ("layers", 1),
                        ("device", torch.device("cpu"))):
        before = getattr(cache, name)
        with pytest.raises(AttributeError, match=name):
            setattr(cache, name, value)
        assert getattr(cache, name) is before
    cache.data[1, 2] = 7                                   # its bytes do
    cache.label = "a user's own"
    cache.label = "and again"


FAR = 1 << 32   # a number that ctypes would cut to its low 32 bits


def test_sizes_beyond_32_bits_are_refused(on_host):
    for page_size, kv_heads, head_dim in ((FAR + 16, 2, 64), (16, FAR + 2, 64), (16, 2, FAR + 64), (16 - FAR, 2, 64)):
        with pytest.raises(ValueError, match="must be 0"):
            qd.KV4Cache(4, page_size, kv_heads, head_dim, device="cpu")
        with pytest.raises(ValueError, match="must be 0"):
            qd.KV4Cache.wrap(torch.zeros((1, 4, 16 * 2 * 72), dtype=torch.uint8), page_size, kv_heads, head_dim)
    cache = qd.KV4Cache(4, 16, 2, 64, device="cpu")
    sizes = dict(rows=8, heads=4, batch=2, max_q_len=4, max_kv_len=4096)
    assert qd.kv4_attention_workspace(cache, **sizes).numel() > 0
    for name in sizes:
        with pytest.raises(ValueError, match=name):
            qd.kv4_attention_workspace(cache, **dict(sizes, **{name: sizes[name] + FAR}))
    assert qd.verify_workspace(2, 3, 100, device="cpu").numel() > 0
    for sizes in ((FAR + 2, 3, 100), (2, FAR + 3, 100), (2, 3, FAR + 100), (2 - FAR, 3, 100)):
        with pytest.raises(ValueError, match="must be 0"):
            qd.verify_workspace(*sizes, device="cpu")
