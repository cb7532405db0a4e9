"""The 8-bit paged cache on the GPU: append, page copies, reading back and
decoding against plain 64-bit references."""
import numpy as np
import pytest
import torch

from content_dependent_block_gb300 import _build, bsa
from tests import attention_reference as att
from tests import paged_reference as ref

pytestmark = pytest.mark.gpu

BF16 = torch.bfloat16


@pytest.fixture(scope="module", autouse=True)
def _lib():
    _build.build()


@pytest.fixture(autouse=True)
def _clean_status():
    bsa.device_status()
    yield
    torch.cuda.synchronize()


def _randn(g, *shape, dtype=BF16):
    return torch.randn(*shape, generator=g).to(dtype)


def _i32(x):
    return torch.as_tensor(x, dtype=torch.int32).cuda()


def _pages8(g, pool, heads, page, d):
    codes = torch.randint(-127, 128, (pool, heads, page, d), generator=g).to(torch.int8)
    return codes, 0.01 + 0.02 * torch.rand(pool, heads, page, generator=g)


class Host:
    """An 8-bit cache on the host and its copy on the device."""

    def __init__(self, g, pool, heads, page, d):
        self.k, self.ks = _pages8(g, pool, heads, page, d)
        self.v, self.vs = _pages8(g, pool, heads, page, d)
        self.kbar = _randn(g, pool, heads, d, dtype=torch.float32)
        self.cache = bsa.PagedCache8(*(x.cuda() for x in (self.k, self.v, self.ks, self.vs, self.kbar)))

    def append(self, new_k, new_v, cu, start, table):
        """Returns the bound on what the means may be off by: n + 2 roundings
        (one more than the products) of the mean of the values' sizes."""
        tol = torch.zeros(self.kbar.shape, dtype=torch.float64)
        self.kbar = self.kbar.double()
        page = self.k.shape[2]
        for s in range(len(start)):
            for i in range(cu[s + 1] - cu[s]):
                p = start[s] + i
                at = (table[s][p // page], slice(None), p % page)
                self.k[at], self.ks[at] = att.quantise(new_k[cu[s] + i])
                self.v[at], self.vs[at] = att.quantise(new_v[cu[s] + i])
            for b in range(start[s] // page, -(-(start[s] + cu[s + 1] - cu[s]) // page)):
                if cu[s + 1] == cu[s]:
                    continue
                rows = min(page, start[s] + cu[s + 1] - cu[s] - b * page)
                at = table[s][b]
                x = att.values(self.k[at, :, :rows], self.ks[at, :, :rows])
                self.kbar[at] = x.mean(1)
                tol[at] = (rows + 2) * 2.0 ** -24 * x.abs().mean(1)
        return tol

    def check(self, tol):
        c = self.cache
        for got, want in ((c.k, self.k), (c.v, self.v), (c.k_scale, self.ks), (c.v_scale, self.vs)):
            assert torch.equal(got.cpu().nan_to_num(-1.0), want.nan_to_num(-1.0))
        ref.assert_within(c.kbar, self.kbar.double(), tol, "means")


@pytest.mark.parametrize("d,page,heads", [(64, 64, 2), (128, 64, 3), (64, 16, 1), (128, 128, 2),
                                          (64, 128, 1), (128, 16, 5), (128, 32, 1), (64, 32, 9)])
@pytest.mark.parametrize("ragged", [True, False])
def test_append(d, page, heads, ragged):
    g = torch.Generator().manual_seed(d + page + heads)
    if ragged:
        new = [1, 0, page - 1, 2 * page + 3, page, 0, 1, 7]
        start = [0, 5, 1, page - 2, 3 * page, 0, page - 1, page]
    else:
        new, start = [3] * 5, [0, page - 1, page - 3, page, 2 * page + 1]
    seqs, width = len(new), 6
    cu = np.cumsum([0] + new).tolist()
    spare = 4 if ragged else 0                   # tokens behind the last sequence
    table = torch.randperm(seqs * width, generator=g).view(seqs, width).tolist()
    host = Host(g, seqs * width + 2, heads, page, d)
    rows = _randn(g, cu[-1] + spare, 2 * heads + 1, d)
    nk, nv = rows[:, :heads], rows[:, heads + 1:]
    on = rows.cuda()
    tol = host.append(nk, nv, cu, start, table)
    for _ in range(2):                           # a call may be repeated
        bsa.cache_append(host.cache, on[:, :heads], on[:, heads + 1:], _i32(table), _i32(start),
                         cu_tokens=_i32(cu) if ragged else None)
        host.check(tol)
    assert bsa.device_status() == 0


@pytest.mark.parametrize("d", [64, 128])
def test_append_rounds_exactly(d):
    """Ties, ratios next to ties, zeros, the smallest and the largest numbers,
    rows that are not finite."""
    g = torch.Generator().manual_seed(d)
    rows = [torch.zeros(d), torch.full((d,), -0.0)]
    for top in (127.0, 63.5, 1.984375, 2.0 ** -120 * 127, 254.0, 1.0, 1.0078125, 255.0):
        # every ratio (2 k + 1) / 254 of a bf16 grid, x = top / 2 among them
        rows.append(torch.cat([torch.tensor([top, -top, top / 2, -top / 2]),
                               top * (2 * torch.randint(-64, 64, (d - 4,), generator=g) + 1) / 254.0]))
    for e in (-133, -130, -126, -120, -7, 0, 8, 100, 127):
        m = torch.randint(1, 256, (d,), generator=g) * torch.randint(-1, 2, (d,), generator=g)
        rows.append(torch.ldexp(m.double(), torch.tensor(e - 8.0)).float() if e > -126 else
                    torch.ldexp(m.double().clamp(-2, 2), torch.tensor(float(e))).float())
    for shrink in range(0, 12):                  # ratios of unlike exponents
        x = _randn(g, d, dtype=torch.float32) * 2.0 ** -shrink
        x[int(torch.randint(0, d, (1,), generator=g))] = 1.0 + shrink / 16
        rows.append(x)
    for bad in (float("inf"), float("-inf"), float("nan")):
        x = _randn(g, d, dtype=torch.float32)
        x[d // 3] = bad
        rows.append(x)
    x = torch.stack(rows).bfloat16()
    x = torch.cat([x, (torch.randint(0, 1 << 16, (200, d), generator=g, dtype=torch.int32) - (1 << 15))
                   .to(torch.int16).view(BF16)])           # any bits
    n = x.shape[0]
    new = x[:, None]
    page = 16
    host = Host(g, -(-n // page), 1, page, d)
    table = [list(range(-(-n // page)))]
    bsa.cache_append(host.cache, new.cuda(), new.flip(0).cuda(), _i32(table), _i32([0]))
    want_k, want_ks = att.quantise(x)
    want_v, want_vs = att.quantise(x.flip(0))
    for got, scale, wc, ws in ((host.cache.k, host.cache.k_scale, want_k, want_ks),
                               (host.cache.v, host.cache.v_scale, want_v, want_vs)):
        assert torch.equal(got.cpu().view(-1, d)[:n], wc)
        s = scale.cpu().view(-1)[:n]
        assert torch.equal(s.isnan(), ws.isnan()) and torch.equal(s[~ws.isnan()], ws[~ws.isnan()])
    # what a row reads back as
    k, v = bsa.cache_read(host.cache, _i32(table), _i32([0]), n)
    for got, wc, ws in ((k, want_k, want_ks), (v, want_v, want_vs)):
        want = (wc.float() * ws[:, None]).bfloat16()
        assert torch.equal(got.cpu()[:, 0].isnan(), want.isnan())
        assert torch.equal(got.cpu()[:, 0].nan_to_num(), want.nan_to_num())
    assert bsa.device_status() == 0


def test_a_row_is_off_by_half_a_step():
    g = torch.Generator().manual_seed(5)
    x = _randn(g, 300, 2, 128)
    cache = bsa.PagedCache8.empty(20, 2, 16, 128)
    table = _i32([list(range(20))])
    bsa.cache_append(cache, x.cuda(), x.cuda(), table, _i32([0]))
    k, v = bsa.cache_read(cache, table, _i32([0]), 300)
    a = x.double().abs().amax(-1, keepdim=True)
    # half a code, the scale's and the product's rounding, the output's
    tol = a / 254 + x.double().abs() * 2.0 ** -22 + 2.0 ** -8 * (x.double().abs() + a / 254)
    ref.assert_within(k, x.double(), tol, "k")
    ref.assert_within(v, x.double(), tol, "v")


@pytest.mark.parametrize("bits", [8, 16])
@pytest.mark.parametrize("d,page,heads", [(64, 64, 2), (128, 16, 3), (128, 128, 1), (64, 32, 5)])
@pytest.mark.parametrize("heads_first", [True, False])
@pytest.mark.parametrize("ragged", [True, False])
def test_read(bits, d, page, heads, heads_first, ragged):
    g = torch.Generator().manual_seed(bits + d + page)
    new = [3, 0, 2 * page + 1, page, 1] if ragged else [page + 5] * 4
    start = [0, 7, page - 1, page, 2 * page + 3][:len(new)]
    cu = np.cumsum([2 if ragged else 0] + new).tolist()      # tokens before the first sequence
    total = cu[-1] + (3 if ragged else 0)                    # and behind the last
    table = torch.randperm(6 * len(new), generator=g).view(len(new), 6).tolist()
    if bits == 8:
        host = Host(g, 6 * len(new), heads, page, d)
        c, val = host.cache, {"k": host.k.float() * host.ks[..., None], "v": host.v.float() * host.vs[..., None]}
    else:
        k, v = _randn(g, 6 * len(new), heads, page, d), _randn(g, 6 * len(new), heads, page, d)
        c = bsa.PagedCache(k.cuda(), v.cuda(), torch.zeros(6 * len(new), heads, d).cuda())
        val = {"k": k, "v": v}
    shape = (heads, total, d) if heads_first else (total, heads, d)
    back = _randn(g, 2, *shape)
    # strided: a slice of a wider tensor
    wide = torch.zeros(2, shape[0], shape[1], d + 8, dtype=BF16, device="cuda")
    wide[..., :d] = back.cuda()
    out = (wide[0, ..., :d], wide[1, ..., :d])
    got = bsa.cache_read(c, _i32(table), _i32(start), total, cu_tokens=_i32(cu) if ragged else None,
                         heads_first=heads_first, out=out)
    want = back.clone()                                      # what no sequence has stays
    for s in range(len(new)):
        for i in range(new[s]):
            p = start[s] + i
            for j, name in enumerate(("k", "v")):
                row = val[name][table[s][p // page], :, p % page].bfloat16()
                if heads_first:
                    want[j, :, cu[s] + i] = row
                else:
                    want[j, cu[s] + i] = row
    for j in range(2):
        assert torch.equal(got[j].cpu(), want[j])
    assert not wide[..., d:].any() and bsa.device_status() == 0


def test_read_reports_and_skips():
    g = torch.Generator().manual_seed(1)
    host = Host(g, 8, 1, 16, 64)
    out = torch.full((2, 96, 1, 64), 7.0, dtype=BF16, device="cuda")
    # page 9 is not there; the second sequence's tokens lie beyond its table
    bsa.cache_read(host.cache, _i32([[0, 9], [1, 2]]), _i32([0, 16]), 64, out=(out[0, :64], out[1, :64]))
    assert bsa.device_status() in (1, 3)                     # whichever CTA came first
    want = (host.k[0].float() * host.ks[0][..., None]).bfloat16().transpose(0, 1)
    got = out[0].cpu()
    assert torch.equal(got[:16], want) and (got[16:32] == 7).all() and (got[64:] == 7).all()
    out.fill_(7.0)
    bsa.cache_read(host.cache, _i32([[0, 1], [1, 2]]), _i32([0, 17]), 64, out=(out[0, :64], out[1, :64]))
    assert bsa.device_status() == 1
    assert (out[:, 32:] == 7).all() and not (out[:, :32] == 7).all()
    bsa.cache_read(host.cache, _i32([[0, 1], [1, 2]]), _i32([-1, 0]), 64, cu_tokens=_i32([0, 40, 20]),
                   out=(out[0, :64], out[1, :64]))
    assert bsa.device_status() == 1


def test_copy_pages():
    g = torch.Generator().manual_seed(2)
    for heads, page, d in ((3, 16, 64), (8, 128, 128)):
        host = Host(g, 40, heads, page, d)
        order = torch.randperm(40, generator=g)
        pairs = torch.stack([order[:17], order[17:34]], 1)
        bsa.copy_pages(host.cache, _i32(pairs))
        for x in (host.k, host.v, host.ks, host.vs, host.kbar):
            x[pairs[:, 1]] = x[pairs[:, 0]]
        host.check(torch.zeros(host.kbar.shape, dtype=torch.float64))
        assert bsa.device_status() == 0
        bsa.copy_pages(host.cache, _i32([[0, 40]]))
        assert bsa.device_status() == 3
        host.check(torch.zeros(host.kbar.shape, dtype=torch.float64))


@pytest.mark.parametrize("d,page,heads,group", [(64, 64, 2, 1), (128, 64, 1, 8), (64, 16, 2, 4), (128, 128, 1, 3),
                                                (128, 32, 2, 16), (64, 32, 1, 7), (128, 16, 1, 20)])
@pytest.mark.parametrize("share", [False, True])
def test_decode(d, page, heads, group, share):
    g = torch.Generator().manual_seed(d + page + group)
    lens = [1, page, 9 * page + 3, 0, 4 * page - 1]
    seqs, width = len(lens), 10
    host = Host(g, seqs * width, heads, page, d)
    table = torch.randperm(seqs * width, generator=g).view(seqs, width)
    # keys as a selection meets them: means that differ; rows past the end hold anything
    val = att.values(host.k, host.ks)
    host.kbar = val.mean(2).float()
    for s, n in enumerate(lens):
        if n % page:
            at = table[s, n // page]
            host.kbar[at] = val[at, :, :n % page].mean(1).float()
            host.ks[at, :, n % page:] = float("nan")
            host.vs[at, :, n % page:] = float("inf")
    c = bsa.PagedCache8(*(x.cuda() for x in (host.k, host.v, host.ks, host.vs, host.kbar)))
    q = _randn(g, seqs, heads * group, d)
    for topk, local in ((3, True), (2, False), (32, True)):
        out, idx = bsa.paged_decode(c, q.cuda(), _i32(table), _i32(lens), topk, local_block=local, share_group=share)
        want, tol, ids = ref.decode(val, att.values(host.v, host.vs), host.kbar, q, table, lens, topk,
                                    local=local, share=share)
        assert torch.equal(idx.cpu(), ids)
        ref.assert_within(out, want, tol, f"decode top-{topk}")
    assert bsa.device_status() == 0


def test_decode_scales_of_every_size():
    """Scales and queries from 2^-120 to 2^90: weights and scores keep within
    their formats."""
    g = torch.Generator().manual_seed(8)
    d, page, seqs = 64, 16, 7
    host = Host(g, seqs * 4, 1, page, d)
    table = torch.arange(seqs * 4).view(seqs, 4)
    q = _randn(g, seqs, 2, d)
    for s, (a, b, c) in enumerate([(0, 0, 0), (-40, 40, 60), (60, -60, -100), (-100, 90, 90), (30, -30, -126),
                                   (0, 0, 100), (90, -100, 20)]):
        host.ks[table[s]] *= 2.0 ** a
        q[s] *= 2.0 ** b
        host.vs[table[s]] *= 2.0 ** c
    host.vs[table[0, :2]] *= 2.0 ** 40            # the largest comes late, and early
    host.vs[table[1, 2:]] *= 2.0 ** 25
    val, vv = att.values(host.k, host.ks), att.values(host.v, host.vs)
    c = bsa.PagedCache8(*(x.cuda() for x in (host.k, host.v, host.ks, host.vs, val.mean(2).float())))
    lens = [64, 60, 64, 33, 64, 50, 64]
    out, idx = bsa.paged_decode(c, q.cuda(), _i32(table), _i32(lens), 4)
    want, tol, ids = ref.decode(val, vv, val.mean(2).float(), q, table, lens, 4)
    assert torch.equal(idx.cpu(), ids)
    tol = tol + _floor(vv, table, lens, page)
    ref.assert_within(out, want, tol, "decode")


def _floor(vv, table, lens, page):
    """Weights in fp16 below its normal range: 2^-37 of the largest scale times
    127 a key, here of the sequence's largest |v|."""
    return torch.stack([n * 2.0 ** -36 * vv[t].abs().amax() for n, t in zip(lens, table)])[:, None, None]


def test_refusals():
    c = bsa.PagedCache8.empty(4, 2, 16, 64)
    with pytest.raises(ValueError):
        bsa.PagedCache8(c.k.float(), c.v, c.k_scale, c.v_scale, c.kbar)
    with pytest.raises(ValueError):
        bsa.PagedCache8(c.k, c.v, c.k_scale[:, :1], c.v_scale, c.kbar)
    with pytest.raises(ValueError):
        bsa.PagedCache8(c.k, c.v, c.k_scale, c.v_scale.double(), c.kbar)
    with pytest.raises(ValueError):
        bsa.PagedCache8(c.k, c.v, c.k_scale, c.v_scale, c.kbar[:, :, :32])
    t, s = _i32([[0]]), _i32([0])
    out = torch.empty(16, 2, 64, dtype=BF16, device="cuda")
    with pytest.raises(bsa.BsaError):                        # one tensor for both
        bsa.cache_read(c, t, s, 16, out=(out, out))
    with pytest.raises(bsa.BsaError):                        # rows overlap
        one = torch.empty(64, dtype=BF16, device="cuda").expand(16, 2, 64)
        bsa.cache_read(c, t, s, 16, out=(one, one))
    with pytest.raises(ValueError):
        bsa.cache_read(c, t, s, 16, out=(out, out.float()))
    with pytest.raises(TypeError):
        bsa.cache_read(c, t, s.long(), 16)
    k, v = bsa.cache_read(c, t, s, 0)
    assert k.shape == (0, 2, 64) and bsa.device_status() == 0
