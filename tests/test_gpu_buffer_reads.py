"""The address check of loads through a buffer address, which ends the reads of
csrc/routed_ffn.hip: a lane reads what lies before the buffer's length, by the
sum of the scalar and the lane's offset, and zeros from there on, with scalar
offsets up to the length itself.  Every address of these calls lies inside the
tensor, whatever the check does."""
import pytest

import mixture_experts_layer_prefix_amd as M
from mixture_experts_layer_prefix_amd import _lib as L

torch = pytest.importorskip("torch")


def check(src, length, scalar, first, lanes):
    got = M.buffer_reads(src, length, scalar, first, lanes)
    a = scalar + first
    want = src[a:a + 16 * lanes].view(torch.int32).view(lanes, 4).clone()
    assert bool((want != 0).all())
    want[max(0, (length - a) // 16):] = 0
    for form, w in zip(got, (want, want, want[:, 0], want[:, 0])):
        assert torch.equal(form, w), (length, scalar, first)


def pattern(n):
    return torch.randint(1, 256, (n,), device="cuda", dtype=torch.uint8, generator=torch.Generator("cuda").manual_seed(1))


@pytest.mark.gpu
@pytest.mark.parametrize("length", [0, 16, 128, 384, 1024, 16384])
def test_reads_end_at_the_length(length):
    """Scalar offsets from zero to the length, lanes that begin before, at and
    behind the end."""
    src = pattern(1 << 16)
    for scalar in sorted({0, 16, 128, length // 32 * 16, length - 16, length}):
        if 0 <= scalar <= length:
            for first in (0, 16, 512, 4096, 16384):
                check(src, length, scalar, first, 64)


@pytest.mark.gpu
def test_reads_end_at_a_length_near_4_gb():
    """Where the sum of both offsets passes 32 bits, as that of scales does
    whose buffer is as long as the routed experts take."""
    length = (1 << 32) - 512
    src = torch.empty(length + (1 << 24), dtype=torch.uint8, device="cuda")
    src[:1 << 16] = pattern(1 << 16)          # where a sum that wraps would read
    src[-(1 << 24) - (1 << 16):] = pattern((1 << 24) + (1 << 16))
    for scalar, first in ((length, 0), (length, 256), (length, 512), (length, 4096), (length, (1 << 24) - 1024),
                          (length - 512, 0), (length - 512, 768), (length - 4096, 3584)):
        check(src, length, scalar, first, 64)


def test_refusals():
    f, fake = L.lib().moe_buffer_reads, 0x100000
    ok = dict(src=fake, bytes=65536, length=1024, scalar=0, first=0, lanes=64, dst=fake)
    for bad in (dict(bytes=1023), dict(bytes=-1), dict(length=65552), dict(scalar=65536), dict(first=65536), dict(lanes=32),
                dict(lanes=-64), dict(lanes=(1 << 24) + 64), dict(scalar=8), dict(first=8), dict(length=8), dict(src=None),
                dict(dst=None), dict(src=fake + 8), dict(dst=fake + 8), dict(bytes=1 << 40, first=(1 << 32) - 1024)):
        a = {**ok, **bad}
        assert f(a["src"], a["bytes"], a["length"], a["scalar"], a["first"], a["lanes"], a["dst"], None) == L.MOE_EINVAL, bad
    assert f(None, 0, 0, 0, 0, 0, None, None) == L.MOE_OK
