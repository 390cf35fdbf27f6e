"""Workspace sizes of the gated delta rule (CPU only)."""
import itertools

import pytest

from test_abi_delta import desc, fwd, need

SEQUENCES = [1, 2, 3, 4, 5, 7, 8, 11, 16, 17, 31, 33, 64, 100, 129, 300]
TOKENS = sorted({t + d for t in (1, 64, 128, 256, 512, 576, 640, 1024, 1152, 1216, 2048, 3000, 4096, 8192, 20000, 65536, 300000)
                 for d in (-1, 0, 1, 64)})


def size(B, H, Hk, T, dk, dv, dtype, keep):
    return need(desc(B=B, H=H, Hk=Hk, T=T, dk=dk, dv=dv, dtype=dtype), keep)


@pytest.mark.parametrize("dtype", [0, 1])
@pytest.mark.parametrize("keep", [0, 1])
@pytest.mark.parametrize("H,Hk,dk,dv", [(16, 16, 128, 128), (1, 1, 64, 64), (4, 2, 32, 80), (6, 2, 64, 96), (3, 1, 128, 16),
                                        (2, 2, 32, 1024), (11, 11, 32, 208)])
def test_a_buffer_for_the_largest_call_serves_smaller_ones(H, Hk, dk, dv, keep, dtype):
    bytes_ = {(B, T): size(B, H, Hk, T, dk, dv, dtype, keep) for B, T in itertools.product(SEQUENCES, TOKENS)
              if B * H * max((T + 63) // 64, (dv + 63) // 64) <= 1 << 22}
    for (B, T), n in bytes_.items():
        assert n > 0 or T == 0
        for less in ((max([b for b in SEQUENCES if b < B], default=B), T), (B, max([t for t in TOKENS if t < T], default=T))):
            assert bytes_[less] <= n, (less, (B, T))


def test_calls_take_what_is_asked_for():
    """... and less is refused."""
    for T in (512, 576, 1152, 1216):
        for dtype in (0, 1):
            d = desc(B=1, H=16, Hk=16, T=T, dk=128, dv=128, dtype=dtype)
            assert fwd(d, wbytes=need(d, 0) - 1) == 4
            assert fwd(desc(B=1, H=16, Hk=16, T=512, dk=128, dv=128, dtype=dtype), wbytes=need(d, 0), o=0x7F0000000000) == 1
