"""Weights in 4 bits at the ends of bf16's range."""
import pytest

import mixture_experts_layer_prefix_amd as M

torch = pytest.importorskip("torch")
from tests import mx_ref as R  # noqa: E402
from tests.test_gpu_mx_ops import BF, U8, I32, check4  # noqa: E402

pytestmark = pytest.mark.gpu


def same(got, codes, scale):
    """got is each value of the codes once rounded to bf16."""
    exact = torch.from_numpy(R.values4(codes.cpu().numpy(), scale.cpu().numpy()))
    want = exact.to(BF)
    assert torch.equal(got.cpu(), want) and torch.equal(got.cpu().signbit(), want.signbit())
    return exact


def test_quantize_up_to_the_largest_finite_value():
    """Every finite bf16 value; blocks that the largest ones lead, which round
    to 2^128 and come back as infinity."""
    v = torch.arange(65536, dtype=I32, device="cuda").to(torch.int16).view(BF)
    v = v[torch.isfinite(v)]
    top = torch.finfo(BF).max
    assert v.numel() % 128 == 0
    check4(v.view(-1, 128).contiguous())
    for lead in (2.0 ** 125, 2.0 ** 126, 2.0 ** 127, 1.5 * 2.0 ** 127, 1.75 * 2.0 ** 127, top):
        some = v[v.abs() <= lead]
        some = torch.cat([some, torch.zeros(-some.numel() % 31, dtype=BF, device="cuda")]).view(-1, 31)
        blocks = torch.cat([torch.full((some.shape[0], 1), lead, dtype=BF, device="cuda"), some], 1)
        blocks = torch.cat([blocks, torch.zeros(-blocks.shape[0] % 4, 32, dtype=BF, device="cuda")]).view(-1, 128)
        check4(blocks)
        back = M.dequantize_mxfp4(*M.quantize_mxfp4(blocks))
        assert bool(torch.isinf(back[0, 0])) == (lead >= 1.75 * 2.0 ** 127)
        # half a step of E2M1 at most: a sixth of the lead
        near = torch.isfinite(back)
        assert bool(((back.double() - blocks.double()).abs()[near] <= lead / 6).all())


@pytest.mark.parametrize("byte", list(range(0, 252, 6)) + [252, 253, 254])
def test_dequantize_is_exact_below_2_128(byte):
    """Every byte of codes at a scale: the value itself, also below bf16's normal
    numbers, and infinity from 2^128 on."""
    codes = torch.arange(256, dtype=U8, device="cuda").view(4, 64)
    scale = torch.full((1, 4, 4), byte, dtype=U8, device="cuda")
    got = M.dequantize_mxfp4(codes, scale)
    exact = same(got, codes, scale)
    finite = exact.abs() < 2.0 ** 128
    assert torch.equal(got.cpu().double()[finite], exact[finite])
    assert bool(torch.isinf(got.cpu()[~finite]).all())
    assert bool(finite.all()) == (byte <= 252)
