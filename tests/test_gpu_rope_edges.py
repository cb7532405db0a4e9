"""Rotary positions on the GPU in sizes that give a thread several heads, in
uneven shares and in more than one batch of loads, against the 64-bit formula
(on the device, so that the sizes cost little)."""
import pytest
import torch

from content_dependent_block_gb300 import _build, bsa
from tests import paged_reference as ref

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    _build.build()


def formula(x, positions, freq, interleaved, factor, sign):
    """(y, tol) in fp64 on x's device; tol as in the CPU reference."""
    half = freq.numel()
    angle = sign * positions.double()[:, None, :, None] * freq.to(x.device)
    c, s = factor * torch.cos(angle), factor * torch.sin(angle)
    y, tol = x.double(), torch.zeros(x.shape, dtype=torch.float64, device=x.device)
    if interleaved:
        ia, ib = slice(0, 2 * half, 2), slice(1, 2 * half, 2)
    else:
        ia, ib = slice(0, half), slice(half, 2 * half)
    a, b = y[..., ia].clone(), y[..., ib].clone()
    y[..., ia], y[..., ib] = a * c - b * s, b * c + a * s
    each = abs(factor) * (a.abs() + b.abs()) * (2.0 ** -21 + angle.abs() * 2.0 ** -51)
    for i in (ia, ib):
        tol[..., i] = each + ref.HALF_STEP[x.dtype] * (y[..., i].abs() + each)
    return y, tol


# heads, n, d, rot, dtype, interleaved: 5 + 5, 7 + 6 and 8 heads of a thread
# for each kernel (halves in vectors, interleaved, halves of any width)
MANY = [
    (10, 20011, 64, 64, torch.bfloat16, False), (13, 20011, 64, 32, torch.bfloat16, False),
    (32, 9801, 64, 64, torch.bfloat16, False), (10, 5003, 128, 128, torch.float32, False),
    (10, 20011, 64, 34, torch.bfloat16, True), (13, 5003, 128, 96, torch.float32, True),
    (32, 9801, 64, 64, torch.bfloat16, True),
    (10, 9901, 64, 34, torch.bfloat16, False), (13, 4999, 128, 34, torch.bfloat16, False),
    (32, 4999, 64, 22, torch.float32, False), (13, 4999, 128, 100, torch.float32, False),
]


@pytest.mark.parametrize("heads,n,d,rot,dtype,inter", MANY)
@pytest.mark.parametrize("way", ["forward", "backward", "in place", "token-major"])
def test_several_heads_of_a_thread(heads, n, d, rot, dtype, inter, way):
    g = torch.Generator(device="cuda").manual_seed(heads + n + rot)
    x = torch.randn(1, n, heads, d, generator=g, device="cuda").to(dtype)
    x = x.transpose(1, 2) if way in ("in place", "token-major") else x.transpose(1, 2).contiguous()
    pos = torch.randint(-9, 40000, (1, n), generator=g, device="cuda", dtype=torch.int32)
    plan = bsa.Rope(rot, interleaved=inter, attention_factor=0.75)
    want, tol = formula(x, pos, ref.inv_freq(rot), inter, 0.75, -1.0 if way == "backward" else 1.0)
    call = bsa.rope_backward if way == "backward" else bsa.rope
    out = x if way == "in place" else torch.empty_like(x) if way == "token-major" else None
    got = call(x, plan, pos, out=out)
    off = (got.double() - want).abs()
    assert bool((off <= tol).all()), float((off - tol).max())


# ------------------------------------------------------------------ autograd
class Turn(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, plan, positions):
        ctx.rest = plan, positions
        return bsa.rope(x, plan, positions)

    @staticmethod
    def backward(ctx, dy):
        return bsa.rope_backward(dy.contiguous(), *ctx.rest), None, None


def test_a_gradient_is_not_dropped_silently():
    plan = bsa.Rope(64)
    x = torch.randn(1, 2, 9, 64, device="cuda", requires_grad=True)
    for call in (bsa.rope, bsa.rope_backward):
        with pytest.raises(ValueError):
            call(x, plan, 3)
        with pytest.raises(ValueError):
            call(x * 2, plan, 3)
        with pytest.raises(ValueError):
            call(x.detach(), plan, 3, out=torch.empty_like(x).requires_grad_())
        with torch.no_grad():
            y = call(x, plan, 3)
        assert torch.equal(y, call(x.detach(), plan, 3)) and not y.requires_grad
    w = torch.randn(1, 2, 9, 64, device="cuda")
    (Turn.apply(x, plan, 3) * w).sum().backward()
    assert torch.equal(x.grad, bsa.rope_backward(w, plan, 3))


def test_tensors_that_autograd_saved_are_not_overwritten_unseen():
    plan = bsa.Rope(64)
    scale = torch.ones(64, device="cuda", dtype=torch.bfloat16, requires_grad=True)
    cache = bsa.PagedCache.empty(4, 2, 16, 64)
    table, ones = (torch.tensor(x, dtype=torch.int32, device="cuda") for x in ([[0], [1]], [1, 1]))
    new = torch.randn(2, 2, 64, device="cuda").bfloat16()
    out, qk = new.clone(), new.transpose(0, 1)
    writes = [
        (qk, lambda: bsa.rope(qk, plan, 1, out=qk)),
        (new, lambda: bsa.rope(qk, plan, 1, out=qk)),                  # the base of a view
        (cache.v, lambda: bsa.cache_append(cache, new, new, table, ones - 1)),
        (cache.k, lambda: bsa.copy_pages(cache, torch.tensor([[0, 2]], dtype=torch.int32, device="cuda"))),
        (out, lambda: bsa.paged_decode(cache, new, table, ones, 1, out=out)),
    ]
    for saved, write in writes:
        y = (saved * scale).sum()
        write()
        with pytest.raises(RuntimeError, match="modified by an inplace operation"):
            y.backward()
        y = (saved * scale).sum()
        y.backward()
    with torch.inference_mode():
        x = torch.randn(2, 9, 64, device="cuda")
        want = bsa.rope(x, plan, 5)
        assert torch.equal(bsa.rope(x, plan, 5, out=x), want)
