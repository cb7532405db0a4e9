"""Rotary positions on the GPU against the 64-bit formula, the gradient
against the formula and against differences, layouts, far positions."""
import pytest
import torch

from content_dependent_block_gb300 import _build, bsa
from tests import paged_reference as ref

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    _build.build()


def _x(shape, dtype, seed=0):
    g = torch.Generator().manual_seed(seed)
    return torch.randn(*shape, generator=g).to(dtype).cuda()


CASES = [  # batch, heads, n, d, rot, dtype, interleaved
    (1, 1, 1, 64, 64, "bf16", False), (1, 3, 7, 128, 128, "bf16", True), (2, 5, 33, 64, 32, "bf16", False),
    (2, 17, 9, 128, 96, "fp32", True), (1, 40, 130, 64, 64, "fp32", False), (3, 2, 65, 64, 16, "fp32", True),
    (1, 4, 31, 64, 2, "bf16", False), (2, 3, 19, 128, 34, "bf16", True), (1, 9, 12, 64, 22, "fp32", False),
    (1, 33, 2049, 128, 128, "bf16", False), (1, 2, 5, 64, 8, "bf16", True),
]


@pytest.mark.parametrize("b,h,n,d,rot,dt,inter", CASES)
@pytest.mark.parametrize("backward", [False, True])
def test_against_the_formula(b, h, n, d, rot, dt, inter, backward):
    dtype = torch.bfloat16 if dt == "bf16" else torch.float32
    x = _x((b, h, n, d), dtype)
    g = torch.Generator().manual_seed(1)
    pos = torch.randint(-5, 3000, (b, n), generator=g, dtype=torch.int32)
    plan = bsa.Rope(rot, interleaved=inter, scaling="linear", factor=2.0, attention_factor=1.25)
    f = bsa.rope_backward if backward else bsa.rope
    y = f(x, plan, pos.cuda())
    want, tol = ref.rope(x, pos, ref.inv_freq(rot, scaling="linear", factor=2.0), inter, 1.25,
                         -1.0 if backward else 1.0)
    ref.assert_within(y, want, tol, "rope")
    assert y.is_contiguous() and y.dtype == dtype
    assert torch.equal(y[..., rot:], x[..., rot:])


@pytest.mark.parametrize("far", [2 ** 20, 2 ** 31 - 1, -2 ** 31])
def test_far_positions_keep_their_angles(far):
    """At 10^6 and beyond an fp32 angle would be off by 0.06 rad and more; the
    tolerance is that of position 0 but for the frequency's own 2^-52."""
    x = _x((1, 2, 16, 128), torch.float32)
    pos = torch.full((1, 16), far, dtype=torch.int32)
    pos -= torch.arange(16, dtype=torch.int32) * (1 if far > 0 else -1)
    plan = bsa.Rope(128)
    want, tol = ref.rope(x, pos, ref.inv_freq(128), False)
    ref.assert_within(bsa.rope(x, plan, pos.cuda()), want, tol, "far")


def test_first_position_and_three_dimensions():
    x = _x((6, 21, 64), torch.bfloat16)
    plan = bsa.Rope(64)
    pos = torch.arange(100, 121, dtype=torch.int32)
    a, b = bsa.rope(x, plan, 100), bsa.rope(x, plan, pos.cuda())
    assert torch.equal(a, b)
    want, tol = ref.rope(x[None], pos[None], ref.inv_freq(64), False)
    ref.assert_within(a[None], want, tol, "3-d")
    own = bsa.Rope(64, inv_freq=ref.inv_freq(64).numpy())
    assert torch.equal(bsa.rope(x, own, 100), a)


@pytest.mark.parametrize("rot", [64, 34])
@pytest.mark.parametrize("inter", [False, True])
def test_layouts_strides_and_in_place(rot, inter):
    """q and k as a projection leaves them side by side, into the forward's
    layout, in place, from a broadcast tensor."""
    qkv = _x((2, 13, 9, 64), torch.bfloat16)               # [batch, n, q + k + v heads, d]
    x = qkv[:, :, :6].transpose(1, 2)
    plan = bsa.Rope(rot, interleaved=inter)
    want = bsa.rope(x.contiguous(), plan, 3)
    assert torch.equal(bsa.rope(x, plan, 3), want)
    out = torch.zeros(2, 13, 9, 64, dtype=torch.bfloat16, device="cuda")
    bsa.rope(x, plan, 3, out=out[:, :, 3:].transpose(1, 2))
    assert torch.equal(out[:, :, 3:].transpose(1, 2), want) and not out[:, :, :3].any()
    keep = qkv.clone()
    bsa.rope(x, plan, 3, out=x)
    assert torch.equal(x, want) and torch.equal(qkv[:, :, 6:], keep[:, :, 6:])
    one = _x((1, 1, 13, 64), torch.bfloat16, 5)
    wide = one.expand(2, 6, 13, 64)
    assert torch.equal(bsa.rope(wide, plan, 3), bsa.rope(wide.contiguous(), plan, 3))


def test_no_tokens():
    x = _x((2, 3, 0, 64), torch.bfloat16)
    assert bsa.rope(x, bsa.Rope(64)).shape == (2, 3, 0, 64)


def test_refused_tensors():
    x = _x((2, 3, 8, 64), torch.bfloat16)
    plan = bsa.Rope(64)
    with pytest.raises(bsa.BsaError):                      # rows of out on top of each other
        bsa.rope(x, plan, out=x[:1, :1].expand(2, 3, 8, 64))
    flat = torch.zeros(2 * 3 * 8 * 64 + 64, dtype=torch.bfloat16, device="cuda")
    a, b = flat[:-64].view(2, 3, 8, 64), flat[64:].view(2, 3, 8, 64)
    with pytest.raises(bsa.BsaError):                      # out is x, shifted
        bsa.rope(a, plan, out=b)
    with pytest.raises(TypeError):
        bsa.rope(x, plan, torch.zeros(8, dtype=torch.int64, device="cuda"))
    with pytest.raises(TypeError):
        bsa.rope(x, plan, torch.zeros(2, 9, dtype=torch.int32, device="cuda"))
    with pytest.raises(TypeError):
        bsa.rope(x.half(), plan)
    with pytest.raises(ValueError):
        bsa.rope(x.transpose(2, 3), plan)
    with pytest.raises(ValueError):
        bsa.rope(x, plan, torch.zeros(2, 8, dtype=torch.int32))


@pytest.mark.parametrize("rot,inter", [(64, False), (32, True), (22, False)])
def test_gradient_against_differences(rot, inter):
    """The map is linear, so a difference quotient of step h has only the
    rounding of two fp32 forward values: 2 * 2^-21 * 2 |x| / h for h = 1 is
    below 2^-18 for |x| <= 4 on unit steps."""
    n = 3
    x = _x((1, 1, n, 64), torch.float32).clamp(-3, 3)
    plan = bsa.Rope(rot, interleaved=inter, attention_factor=1.5)
    w = _x((1, 1, n, 64), torch.float32, 7)
    dx = bsa.rope_backward(w, plan, 50)
    base = bsa.rope(x, plan, 50).double()
    for j in range(0, 64, 5):
        for i in range(n):
            y = x.clone()
            y[0, 0, i, j] += 1.0
            step = float(y[0, 0, i, j].double() - x[0, 0, i, j].double())
            diff = float(((bsa.rope(y, plan, 50).double() - base) * w.double()).sum() / step)
            # at most two outputs differ, each by |w| 2^-18
            assert abs(diff - float(dx[0, 0, i, j])) <= 2.0 ** -17 * (float(w.abs().max()) + 1)


def test_backward_undoes_forward_up_to_the_factor():
    x = _x((1, 4, 50, 128), torch.float32)
    plan = bsa.Rope(128, attention_factor=2.0)
    y = bsa.rope_backward(bsa.rope(x, plan, 1 << 20), plan, 1 << 20)
    # two rotations, each off by 2^-21 (|a| + |b|) m, plus fp32 roundings
    assert float((y - 4 * x).abs().max()) <= 2 * 4 * 2.0 ** -20 * 2 * float(x.abs().max())


def test_streams_and_graph_replay():
    x = _x((2, 4, 300, 64), torch.bfloat16)
    plan = bsa.Rope(64)
    pos = torch.arange(600, dtype=torch.int32, device="cuda").view(2, 300)
    want = bsa.rope(x, plan, pos)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        got = bsa.rope(x, plan, pos)
    side.synchronize()
    assert torch.equal(got, want)
    out, dx = torch.zeros_like(x), torch.zeros_like(x)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        bsa.rope(x, plan, pos, out=out)
        bsa.rope_backward(out, plan, pos, out=dx)
    x.copy_(_x((2, 4, 300, 64), torch.bfloat16, 9))
    pos += 77
    g.replay()
    assert torch.equal(out, bsa.rope(x, plan, pos))
    assert torch.equal(dx, bsa.rope_backward(out, plan, pos))
