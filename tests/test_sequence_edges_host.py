"""The sequence operators' binding without a GPU: calls that are refused."""
import pytest
import torch

import device_wide_prefix_tile_amd as dw
from device_wide_prefix_tile_amd import sequence as seq


def test_tensors_that_require_gradients_are_refused():
    """Nothing is recorded for autograd: where it records, such a tensor is refused; elsewhere it is data."""
    x, w = torch.zeros(1, 4, 8), torch.zeros(8, 4)
    tok, table = torch.zeros(3, dtype=torch.int32), torch.zeros(4, 8)
    for t, call in ((x, lambda: dw.causal_conv1d(x, w)), (x, lambda: dw.selective_scan(x, x, w, x[:, :, None, :4], x[:, :, None, :4])),
                    (x[:, 0], lambda: dw.causal_conv1d_step(x[:, 0], x[:, :3], w))):
        x.requires_grad_()
        with pytest.raises(ValueError, match="requires a gradient"):
            call()
        with torch.no_grad(), pytest.raises(ValueError, match="device tensor"):  # the next check
            call()
        x.requires_grad_(False)
        with pytest.raises(ValueError, match="device tensor"):
            call()
    p = torch.nn.Parameter(w)
    for check in (lambda t: seq._plain(t, "weight", (8, 4), torch.float32, -1), lambda t: seq._like(t, "B", (8, 4), torch.float32, -1, 4)):
        with pytest.raises(ValueError, match="weight.detach|B.detach"):
            check(p)
        check(p.detach())
        with torch.no_grad():
            check(p)
    with pytest.raises(ValueError, match="device tensor"):
        dw.embedding_lookup(tok, table)


def test_no_sequences_with_offsets_is_a_call():
    """Offsets of no sequence leave every row outside; without offsets rows need a sequence."""
    import ctypes

    L = seq._lib()
    mb = 1 << 20  # fake device addresses: only sizes are asked for
    args = dict(dtype=0, rows=64, seqs=0, channels=8, states=16, groups=1, x=mb, x_stride=8, delta=2 * mb, delta_stride=8, A=3 * mb,
                B=4 * mb, b_stride=16, C=5 * mb, c_stride=16)
    conv = dict(dtype=0, weight_dtype=0, width=4, rows=64, seqs=0, channels=8, x=mb, x_stride=8, weight=2 * mb)
    for offsets, there in ((6 * mb, True), (None, False)):
        assert (L.selective_scan_workspace(ctypes.byref(seq._ScanArgs(seq_offsets=offsets, **args))) > 0) == there
        assert (L.causal_conv1d_grad_workspace(ctypes.byref(seq._ConvArgs(seq_offsets=offsets, **conv))) > 0) == there
