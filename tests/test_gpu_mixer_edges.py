"""The token mixers at the edges of what their entry points accept: offsets that
name more rows than there are, an epsilon of zero, values that are not finite,
workspaces shared by calls of different sizes."""

import struct

import pytest
import torch

from test_gpu_mixers import BF, DEV, lin_inputs

pytestmark = pytest.mark.gpu


def view4(t):
    return struct.pack("Pqqq", t.data_ptr(), *t.stride()[:3])


@pytest.mark.parametrize("T,H,D,times", [(8192, 2, 64, 2), (65536, 1, 128, 4), (16384, 3, 128, 15)])
def test_linattn_overlapping_offsets_stay_in_the_workspace(lib, T, H, D, times):
    """Offsets 0, T, 0, T, ...: every second sequence holds the whole row, so that
    their segments add up to more than the workspace has room for. The status
    says so, and what lies past the workspace's reported size is left alone."""
    cu = torch.tensor([0, T] * times, dtype=torch.int32, device=DEV)
    n = 2 * times - 1
    q, k, v, do, _, _ = lin_inputs(1, T, H, D, D, BF, T + H, n=n, state=False)
    g = torch.full((H,), -0.01, device=DEV)
    size = lib.linattn_workspace_bytes(1, T, H, D, D, n)
    past = 3 * times * (T // 128) * H * D * D * 4  # every segment of four chunks that the offsets name, and more
    buf = torch.full((size + past,), 0x5a, dtype=torch.uint8, device=DEV)
    o, dq, dk, dv = (torch.empty_like(t) for t in (v, q, k, v))
    hT, dh0 = (torch.empty(n, H, D, D, device=DEV) for _ in range(2))
    raw, s = lib.lib(), torch.cuda.current_stream().cuda_stream
    for run in ("fwd", "bwd"):
        assert raw.scan_workspace_init(buf.data_ptr(), size, s) == lib.SCAN_OK
        if run == "fwd":
            st = raw.linattn_fwd(view4(q), view4(k), view4(v), g.data_ptr(), None, cu.data_ptr(), n, view4(o),
                                 hT.data_ptr(), 1, T, H, D, D, 1.0, lib.SCAN_BF16, buf.data_ptr(), size, s)
        else:
            st = raw.linattn_bwd(view4(q), view4(k), view4(v), g.data_ptr(), None, cu.data_ptr(), n, view4(do),
                                 hT.data_ptr(), view4(dq), view4(dk), view4(dv), dh0.data_ptr(), 1, T, H, D, D, 1.0,
                                 lib.SCAN_BF16, buf.data_ptr(), size, s)
        assert st == lib.SCAN_OK
        assert raw.scan_get_device_status(buf.data_ptr(), s) == lib.SCAN_ERR_SEQLENS
        assert bool((buf[size:] == 0x5a).all()), run
