"""The binding's workspaces and device findings, without a GPU: the library's
calls are replaced by a note of what they were given."""

import weakref

import pytest
import torch

import associative_affine_scan_gb300 as scan
from associative_affine_scan_gb300 import _binding


@pytest.fixture(scope="module", autouse=True)
def built():
    from associative_affine_scan_gb300 import build_lib
    build_lib.build()


@pytest.mark.parametrize("name", ["qk_norm_rope_bwd", "linattn_fwd", "linattn_bwd", "window_attn_fwd",
                                  "window_attn_bwd"])
def test_workspace_lives_until_the_call_has_returned(monkeypatch, name):
    """Another thread may grow the pool's buffer between a call's look-up and its
    launch: the call itself has to hold what it was given."""
    given = []

    def get(nbytes, device, stream):
        buf = torch.empty(nbytes, dtype=torch.uint8)
        given.append((weakref.ref(buf), buf.data_ptr(), buf.numel()))
        return buf

    def enter(device, where, *args):
        buf, at, size = given.pop()
        assert where == name and buf() is not None
        offset = 256 if name.startswith("qk") else 0
        assert (at + offset, size - offset) in list(zip(args, args[1:]))

    monkeypatch.setattr(_binding, "_heads", lambda t, *a, **k: t)
    monkeypatch.setattr(_binding, "_need", lambda t, *a, **k: t)
    monkeypatch.setattr(_binding, "_raw_stream", lambda stream, device: 0)
    monkeypatch.setattr(_binding._mixer_ws, "get", get)
    monkeypatch.setattr(_binding, "_enter", enter)
    x, g = torch.zeros(1, 8, 2, 64), torch.zeros(2)
    {"qk_norm_rope_bwd": lambda: scan.qk_norm_rope_bwd(x, x, None, None, None, None, x, x),
     "linattn_fwd": lambda: scan.linattn_fwd(x, x, x, g),
     "linattn_bwd": lambda: scan.linattn_bwd(x, x, x, g, x),
     "window_attn_fwd": lambda: scan.window_attn_fwd(x, x, x, 4),
     "window_attn_bwd": lambda: scan.window_attn_bwd(x, x, x, x, torch.zeros(1, 2, 8), x, 4)}[name]()
    assert not given


@pytest.mark.parametrize("captured", [False, True])
def test_a_larger_workspace_leaves_the_captured_one(monkeypatch, captured):
    """A graph writes into the workspace of its capture whenever it is replayed:
    the buffer stays when later calls need larger ones. Any other goes when the
    next one is replaced."""
    import ctypes
    monkeypatch.setattr(_binding, "_call", lambda *a: scan.SCAN_OK)
    monkeypatch.setattr(_binding.torch.cuda, "synchronize", lambda device: None)
    monkeypatch.setattr(_binding.torch.cuda, "is_current_stream_capturing", lambda: capturing)
    pool, dev, s = _binding._Workspaces(), torch.device("cpu"), ctypes.c_void_p(3)
    capturing = False
    first = weakref.ref(pool.get(5000, dev, s))
    capturing = captured
    assert pool.get(4000, dev, s) is first()
    capturing = False
    other = weakref.ref(pool.get(5000, dev, ctypes.c_void_p(4)))
    second = weakref.ref(pool.get(9000, dev, s))
    assert pool.get(9000, dev, s) is second() and first() is not None
    pool.get(20000, dev, s)
    assert second() is not None and (first() is not None) == captured
    pool.get(30000, dev, s)
    pool.get(20000, dev, ctypes.c_void_p(4))
    pool.get(30000, dev, ctypes.c_void_p(4))
    assert second() is None and other() is None and (first() is not None) == captured


def test_a_replaced_workspace_stays_while_a_call_holds_it(monkeypatch):
    """A thread between its look-up and its launch, while others need ever larger
    buffers: its own goes only with a wait for the device that comes after."""
    import ctypes
    monkeypatch.setattr(_binding, "_call", lambda *a: scan.SCAN_OK)
    monkeypatch.setattr(_binding.torch.cuda, "is_current_stream_capturing", lambda: False)
    pool, dev, s = _binding._Workspaces(), torch.device("cpu"), ctypes.c_void_p(3)
    waits = []
    monkeypatch.setattr(_binding.torch.cuda, "synchronize", lambda device: waits.append(mine() is not None))
    mine = lambda: None  # noqa: E731
    handed = pool.get(5000, dev, s)
    mine = weakref.ref(handed)
    for n in range(2, 6):
        pool.get(5000 * n, dev, s)
    del handed  # the launch has been made
    assert mine() is not None
    pool.get(40000, dev, s)
    assert waits == [False] + [True] * 5 and mine() is None


def test_no_finding_is_lost(monkeypatch):
    """The scans' workspace, the mixers' and one that a graph still uses have a
    status word each: as many calls as there are findings return them all."""
    import ctypes
    dev, s = torch.device("cpu"), ctypes.c_void_p(3)
    bufs = [torch.empty(16, dtype=torch.uint8) for _ in range(3)]
    found = {b.data_ptr(): f for b, f in zip(bufs, (scan.SCAN_ERR_SEQLENS, scan.SCAN_ERR_TIMEOUT,
                                                    scan.SCAN_ERR_SEQLENS))}

    def call(device, name, ptr, stream):
        assert name == "scan_get_device_status"
        return found.pop(ptr.value, scan.SCAN_OK)

    monkeypatch.setattr(_binding, "_call", call)
    monkeypatch.setattr(_binding, "_stream", lambda stream, device: s)
    for pool, buf in ((_binding._ws, bufs[0]), (_binding._mixer_ws, bufs[1])):
        monkeypatch.setitem(pool._buf, (None, 3), buf)
    monkeypatch.setattr(_binding._mixer_ws, "_held", {(None, 3): [bufs[2]]}, raising=False)
    assert [scan.scan_get_device_status(dev) for _ in range(4)] == [
        scan.SCAN_ERR_SEQLENS, scan.SCAN_ERR_TIMEOUT, scan.SCAN_ERR_SEQLENS, scan.SCAN_OK]


def test_packed_rows_that_are_not_cut_need_no_states():
    """Many sequences fill the GPU uncut: room for the status word, not for a state
    of every sequence and head (4000 x 16 x 128 x 128 fp32, three passes: 12.6 GB).
    Few are cut: room for their segments' states, and no more."""
    assert scan.linattn_workspace_bytes(1, 4000 * 200, 16, 128, 128, 4000) == 256
    assert scan.linattn_workspace_bytes(1, 500, 1, 128, 128, 1) == 256
    assert 256 < scan.linattn_workspace_bytes(1, 60000, 16, 128, 128, 3) < 1 << 28


def test_packed_segments_have_32_bit_lengths():
    """Rows of close to 2^31 steps are cut where many sequences would leave them
    whole: the kernels count a segment's steps in 32 bits."""
    for T in (2 ** 31 - 1, 2 ** 31 - 128, 2 ** 30):
        assert scan.linattn_workspace_bytes(1, T, 1, 8, 8, 400) >= 256 + 3 * (T >> 27) * 8 * 8 * 4
    assert scan.linattn_workspace_bytes(1, 2 ** 27, 1, 8, 8, 400) == 256
