"""sage_rope and sage_rope_tables against cos and sin in 64 bits."""
import numpy as np
import pytest
import torch

import bit_quantized_attention_sage_b200 as sage
import cache_ref as ref

pytestmark = pytest.mark.gpu
DTS = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}


def check(x, y, positions, f, layout, amp, inverse):
    """cos and sin of an angle reduced in fp64: the fraction's fp32 rounding
    (2^-25 of half a turn, so pi 2^-24) and sincospif's 2 units; then three
    fp32 roundings of terms up to amp (|x0| + |x1|); half a step of the type."""
    want = ref.rope(x, positions, f, layout, amp, inverse)
    R = 2 * len(f)
    mag = np.abs(ref.rope(x, positions, np.zeros(R // 2), layout, 1.0, False))
    other = mag.copy()
    i = slice(0, R // 2) if layout == "half" else slice(0, R, 2)
    j = slice(R // 2, R) if layout == "half" else slice(1, R, 2)
    other[..., i], other[..., j] = mag[..., j], mag[..., i]
    both = mag + other
    tol = amp * both * (np.pi * 2.0 ** -24 + 8 * 2.0 ** -24) + ref.half_step(want, x.dtype) * 1.001 + \
        torch.finfo(x.dtype).tiny
    got = y.double().cpu().numpy()
    assert (np.abs(got - want)[..., :R] <= tol[..., :R]).all()
    assert np.array_equal(got[..., R:], x.double().cpu().numpy()[..., R:])


@pytest.mark.parametrize("layout", ["half", "interleaved"])
@pytest.mark.parametrize("dt", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("B,H,N,D,R", [(1, 1, 1, 128, 128), (2, 3, 17, 64, 64), (2, 5, 40, 128, 64),
                                       (1, 2, 33, 128, 6), (3, 2, 5, 96, 80), (1, 1, 3, 7, 2),
                                       (2, 2, 4, 64, 0)])
def test_rope(layout, dt, B, H, N, D, R):
    g = torch.Generator().manual_seed(R + N)
    x = torch.randn((B, H, N, D), generator=g).to(DTS[dt]).cuda()
    pos = torch.randint(0, 10 ** 6, (B, N), generator=g)
    f = torch.tensor([10000.0 ** (-2.0 * p / max(R, 1)) for p in range(R // 2)], dtype=torch.float64)
    for inverse in (False, True):
        y = sage.rope(x, pos.cuda(), f.cuda(), layout=layout, amplitude=1.2, inverse=inverse)
        check(x, y, pos, f.numpy(), layout, 1.2, inverse)
    p32 = pos[0].to(torch.int32).cuda()  # shared int32 positions, in place
    z = x.clone()
    assert sage.rope(z, p32, f.cuda(), layout=layout, out=z) is z
    check(x, z, pos[:1].expand(B, N), f.numpy(), layout, 1.0, False)


@pytest.mark.parametrize("scaling", [None, ("linear", 4.0), ("ntk", 8.0), ("yarn", 8.0, 4096),
                                     ("yarn", 4.0, 8192, 20.0, 2.0)])
def test_rope_far_positions(scaling):
    # a position far out keeps its phase: the angle is some 10^9 radians
    f, amp = sage.rope_freqs(64, scaling=scaling)
    x = torch.randn((1, 2, 3, 64), generator=torch.Generator().manual_seed(1)).cuda()
    pos = torch.tensor([[10 ** 9, 10 ** 9 + 1, 123456789]])
    y = sage.rope(x, pos.cuda(), f, amplitude=amp)
    check(x, y, pos, f.cpu().numpy(), "interleaved", amp, False)


def test_rope_strides():
    f, _ = sage.rope_freqs(64)
    g = torch.Generator().manual_seed(2)
    base = torch.randn((2, 19, 4, 67), generator=g).to(torch.bfloat16).cuda()
    pos = torch.arange(19)[None].expand(2, 19)
    for x in (base[..., :64].transpose(1, 2), base[..., 3:].transpose(1, 2),
              base[:1, :, :1, :64].transpose(1, 2).expand(2, 4, 19, 64)):
        y = sage.rope(x, pos.contiguous().cuda(), f, layout="half")
        check(x, y, pos, f.cpu().numpy(), "half", 1.0, False)


def test_inverse_is_the_gradient():
    # <rope(x), dy> = <x, rope^T(dy)> and, being linear, its differences
    f, amp = sage.rope_freqs(48, scaling=("yarn", 8.0, 100))
    g = torch.Generator().manual_seed(3)
    x, dy = (torch.randn((1, 2, 30, 64), generator=g).cuda() for _ in range(2))
    pos = torch.arange(30, device="cuda") * 7
    for layout in ("half", "interleaved"):
        y = sage.rope(x, pos, f, layout=layout, amplitude=amp).double()
        dx = sage.rope(dy, pos, f, layout=layout, amplitude=amp, inverse=True).double()
        a, b = (y * dy.double()).sum(), (x.double() * dx).sum()
        assert abs(a - b) <= 64 * 2.0 ** -24 * amp * (x.double().abs() * dy.double().abs()).sum()
        for at in ((0, 0, 3, 1), (0, 1, 29, 25), (0, 0, 7, 60)):
            e = torch.zeros_like(x)
            e[at] = 1.0
            step = sage.rope(x + e, pos, f, layout=layout, amplitude=amp).double() - y
            assert abs((step * dy.double()).sum() - dx[at]) <= 1e-4


def test_tables_drive_the_quantizer():
    # quant_qk with rope_tables rotates as rope does (up to rope's rounding of
    # its fp32 result): the same angles in both
    from bit_quantized_attention_sage_b200 import synth
    f, amp = sage.rope_freqs(64, scaling=("yarn", 4.0, 1000))
    pos = torch.arange(5000, 5200, device="cuda")
    c, s = sage.rope_tables(pos, f, amp)
    ang = pos.double()[:, None] * f
    assert (c.double() - torch.cos(ang) * amp).abs().max() <= amp * 12 * 2.0 ** -24
    assert (s.double() - torch.sin(ang) * amp).abs().max() <= amp * 12 * 2.0 ** -24
    x = torch.randn((1, 2, 200, 64), generator=torch.Generator().manual_seed(4)).to(torch.bfloat16).cuda()
    q8 = sage.quant_qk(x, x, x, rope=(c, s, c, s))
    y = sage.rope(x.float(), pos, f, amplitude=amp)
    deq = q8.view("q_i8").float() * q8.view("q_scale").repeat_interleave(64, -1)[..., None]
    step = q8.view("q_scale").repeat_interleave(64, -1)[:, :, :200, None]
    assert ((deq[:, :, :200] - y).abs() <= 0.5001 * step + 1e-5).all()
    assert sage.sync_status() == 0
