"""Sampling from logits with NaN of every kind: quiet, signalling, with a sign."""
import pytest
import torch

import device_wide_prefix_tile_amd as dw

pytestmark = pytest.mark.gpu

T = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}


QUIET, SIGNALLING = {"f32": 0x7FC00001, "f16": 0x7E01, "bf16": 0x7FC1}, {"f32": 0x7F800001, "f16": 0x7C01, "bf16": 0x7F81}


def with_bits(z, where, bits):
    """z with the values of `where` replaced by that bit pattern."""
    i = z.clone().view(torch.int32 if z.dtype == torch.float32 else torch.int16)
    i[where] = bits
    return i.view(z.dtype)


@pytest.mark.parametrize("t", list(T))
def test_signalling_nan_is_as_quiet_nan(t):
    """Neither is ever taken, whatever sign and bits it has: alone in a row, alone in a group of pieces, beside others."""
    g = torch.Generator(device="cuda").manual_seed(5)
    n = 20000
    z, u = (torch.randn(6, n, generator=g, device="cuda") * 2).to(T[t]), torch.zeros(6, device="cuda")
    where = torch.zeros(6, n, dtype=torch.bool, device="cuda")
    where[0] = True
    where[1, :n // 2] = True
    where[2, n // 2:] = True
    where[3, ::2] = True
    where[4, 1:] = True
    where[5, 8192:16384] = True
    kinds = [QUIET[t], SIGNALLING[t], SIGNALLING[t] - (1 << 31 if t == "f32" else 1 << 15)]  # the last one: with a sign
    for s in (dict(), dict(temperature=0.0), dict(top_k=40), dict(top_k=3000), dict(top_p=0.9), dict(min_p=0.02), dict(top_k=2000, top_p=0.7, min_p=0.01)):
        for value in (0.0, 0.5, 1.0 - 2.0 ** -24):
            v = torch.full_like(u, value)
            got = [dw.sample_tokens(with_bits(z, where, bits), v, **s) for bits in kinds]
            assert torch.equal(got[0], got[1]) and torch.equal(got[0], got[2]), (s, value, got)
            assert int(got[0][0]) == -1 and int(got[0][4]) == 0 and not where[torch.arange(1, 6, device="cuda"), got[0][1:].long()].any()
