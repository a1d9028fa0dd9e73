"""GPU parity of the grouped gated norm against the fp64 oracle.

Tolerances: float32 inside -- the sums of at most 8192 squares (pairwise over
lanes: below 20 u, u = 2^-24), rsqrt and SiLU of a few 2^-22 each: relative
2e-6 of a value, of which n w + b may cancel (elements are held against the
rms); outputs rounded once, half a step of the type: a bf16 value 1.f has 7
fraction bits, so steps of 2^-7 of its power of two and a half step of up to
2^-8 of the value.
"""
import numpy as np
import pytest
import torch

import oracle

from gpu_util import Guarded

pytestmark = pytest.mark.gpu


def make(rows, C, io, seed=1):
    g = torch.Generator().manual_seed(seed)
    dt = torch.float32 if io == "f32" else torch.bfloat16
    # groups of different size and offset
    x = (torch.randn(rows, C, generator=g) * torch.exp(torch.randn(1, C, generator=g)) + 0.5).to(dt)
    return x, torch.randn(rows, C, generator=g).to(dt) * 2, 1 + torch.randn(C, generator=g), torch.randn(C, generator=g)


def close(got, ref, io, what):
    got, ref = np.asarray(got, np.float64), np.asarray(ref, np.float64)
    assert np.all(np.isfinite(got)), what
    rms = np.sqrt(np.mean(ref * ref)) if ref.size else 1.0
    tol = 8e-6 * np.maximum(rms, np.abs(ref)) + (2 ** -8 * np.abs(ref) if io == "bf16" else 0)
    bad = np.abs(got - ref) > tol
    assert not bad.any(), f"{what}: {int(bad.sum())} elements, worst {np.max(np.abs(got - ref) / tol):.3g} of the bound"


@pytest.mark.parametrize("io", ["bf16", "f32"])
@pytest.mark.parametrize("kind", ["rms", "group"])
@pytest.mark.parametrize("gate", [None, "after", "before"])
@pytest.mark.parametrize("rows, C, D", [(1, 8, 8), (3, 24, 8), (37, 96, 32), (5, 160, 40), (9, 4096, 128), (6, 768, 256),
                                        (4, 1000, 1000), (3, 2560, 1280), (2, 4096, 4096), (3, 8192, 8192), (2, 7680, 1920)])
def test_shapes(cuda_lib, io, kind, gate, rows, C, D):
    from selective_state_space_52_b200 import axon_ssm
    x, z, w, b = make(rows, C, io)
    for shared in (False, True):
        w1, b1 = (w[:D], b[:D]) if shared else (w, b)
        out = Guarded((rows, C), x.dtype)
        axon_ssm.gated_norm(x.cuda(), w1.cuda(), None if gate is None else z.cuda(), bias=b1.cuda(), group=D, kind=kind,
                            gate=gate or "after", out=out.t)
        torch.cuda.synchronize()
        assert out.canaries_intact()
        ref = oracle.gated_norm(x, D, kind, gate, True, z, w1, b1)
        close(out.t.float().cpu(), ref, io, f"{io} {kind} {gate} {rows}x{C}/{D} shared {shared}")


@pytest.mark.parametrize("gate", [None, "after", "before"])
def test_without_activation_weight_bias(cuda_lib, gate):
    from selective_state_space_52_b200 import axon_ssm
    x, z, _, _ = make(11, 256, "f32")
    got = axon_ssm.gated_norm(x.cuda(), None, None if gate is None else z.cuda(), group=64, act=False, eps=1e-3,
                              gate=gate or "after")
    close(got.cpu(), oracle.gated_norm(x, 64, "rms", gate, False, z, eps=1e-3), "f32", str(gate))


@pytest.mark.parametrize("io", ["bf16", "f32"])
def test_row_strides_and_in_place(cuda_lib, io):
    """x and z as slices of one projected row, the result over x: what lies
    beside the slices stays."""
    from selective_state_space_52_b200 import axon_ssm
    x, z, w, _ = make(21, 512, io)
    pad = torch.full((21, 16), 9.0, dtype=x.dtype)
    row = torch.cat([pad, x, pad, z, pad], 1).cuda()
    xs, zs = row[:, 16:528], row[:, 544:1056]
    want = axon_ssm.gated_norm(x.cuda(), w.cuda(), z.cuda(), group=128)
    got = axon_ssm.gated_norm(xs, w.cuda(), zs, group=128)
    assert got.is_contiguous() and torch.equal(got, want)
    axon_ssm.gated_norm(xs, w.cuda(), zs, group=128, out=xs)
    assert torch.equal(xs, want) and torch.equal(zs, z.cuda())
    assert all((row[:, a:a + 16] == 9).all() for a in (0, 528, 1056))
    z2 = z.cuda()
    axon_ssm.gated_norm(x.cuda(), w.cuda(), z2, group=128, out=z2)
    assert torch.equal(z2, want)


def test_offset_far_above_the_spread(cuda_lib):
    """Group norm of values around 1000 with spread 1: the mean leaves before
    the squares are summed (float32 inputs carry the values to 2^-14 of the
    spread, which both sides see alike)."""
    from selective_state_space_52_b200 import axon_ssm
    g = torch.Generator().manual_seed(3)
    x = 1000 + torch.randn(7, 1024, generator=g)
    got = axon_ssm.gated_norm(x.cuda(), group=256, kind="group", act=False).cpu().numpy()
    ref = oracle.gated_norm(x, 256, "group", None, False)
    # the mean is off by at most 2^-24 * 1000 * a few = 2e-4 of the spread
    assert np.max(np.abs(got - ref)) <= 3e-4


def test_zero_rows_and_stream(cuda_lib):
    from selective_state_space_52_b200 import axon_ssm
    x, z, w, _ = make(300, 1024, "bf16")
    assert axon_ssm.gated_norm(x[:0].cuda(), group=128).shape == (0, 1024)
    zero = axon_ssm.gated_norm(torch.zeros(4, 256, device="cuda"), group=64)
    assert torch.equal(zero, torch.zeros_like(zero))
    xc, zc, wc = x.cuda(), z.cuda(), w.cuda()
    want = axon_ssm.gated_norm(xc, wc, zc, group=128)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = axon_ssm.gated_norm(xc, wc, zc, group=128, stream=side)
    side.synchronize()
    assert torch.equal(got, want)


@pytest.mark.parametrize("D", [64, 1920])
def test_infinity_stays_in_its_group(cuda_lib, D):
    """A group with a NaN or an infinity does not touch its neighbours."""
    from selective_state_space_52_b200 import axon_ssm
    x = torch.randn(33, 4 * D, device="cuda", generator=torch.Generator("cuda").manual_seed(5))
    want = axon_ssm.gated_norm(x, group=D, kind="group")
    bad = x.clone()
    bad[3, D] = float("nan")
    bad[32, 4 * D - 1] = float("inf")
    got = axon_ssm.gated_norm(bad, group=D, kind="group")
    touched = torch.zeros_like(x, dtype=torch.bool)
    touched[3, D:2 * D] = touched[32, 3 * D:] = True
    assert got[touched].isnan().all()
    assert torch.equal(got[~touched], want[~touched])
