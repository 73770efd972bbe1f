"""Embedding lookup and its gradient. The lookup is one product rounded once;
the gradient is scale * the canonical tree over a token's rows in order, so
both are compared bit for bit with the oracle's reduction."""
import numpy as np
import pytest
import torch

import oracle

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
TYPES = [torch.float32, torch.bfloat16, torch.float16]


@pytest.fixture(scope="module")
def scr():
    import scan_canonical_reduce_gb300 as m
    return m


def gen(seed):
    return torch.Generator().manual_seed(seed)


def skewed(n, V, seed, pad=0.05):
    g = gen(seed)
    t = (torch.exp(torch.rand(n, generator=g, dtype=torch.float64) * np.log(V)) - 1).long()
    t = t.clamp(0, V - 1) * 7919 % V
    t[torch.rand(n, generator=g) < pad] = -1
    t[torch.rand(n, generator=g) < pad / 2] = V + 3
    return t


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("n,V,D", [(1, 1, 1), (5, 100, 1024), (33, 7, 77), (300, 1000, 130),
                                   (257, 50, 2056), (0, 10, 16), (4, 10, 0)])
@pytest.mark.parametrize("index", [torch.int32, torch.int64])
def test_lookup(scr, dtype, n, V, D, index):
    table = torch.randn(V, D, generator=gen(1)).to(dtype)
    tok = skewed(n, V, 2)
    got = scr.embedding(tok.to(index).to(DEV), table.to(DEV), 1.7)
    ok = (tok >= 0) & (tok < V)
    want = table[tok.clamp(0, V - 1)].float() * torch.tensor(1.7, dtype=torch.float32)
    want = torch.where(ok[:, None], want, 0.0).to(dtype)
    assert got.dtype == dtype and torch.equal(got.cpu(), want)


def test_lookup_shapes_and_strides(scr):
    table = torch.randn(40, 64, generator=gen(3)).to(torch.bfloat16).to(DEV)
    tok = torch.randint(0, 40, (3, 5), generator=gen(4)).to(DEV)
    want = (table[tok].float() * 0.5).to(torch.bfloat16)
    assert torch.equal(scr.embedding(tok, table, 0.5), want)
    # a table whose rows start off 16 bytes, one that is transposed, tokens in steps
    odd = torch.zeros(40, 67, dtype=torch.bfloat16, device=DEV)[:, 3:]
    odd.copy_(table)
    assert torch.equal(scr.embedding(tok, odd, 0.5), want)
    assert torch.equal(scr.embedding(tok, table.t().contiguous().t(), 0.5), want)
    wide = torch.zeros(3, 10, dtype=torch.int64, device=DEV)
    wide[:, ::2] = tok
    assert torch.equal(scr.embedding(wide[:, ::2], table, 0.5), want)
    out = torch.full((16, 70), float("nan"), dtype=torch.bfloat16, device=DEV)
    r = scr.embedding(tok.flatten(), table, 0.5, out=out[:15, 1:65])
    assert torch.equal(r, want.view(15, 64))
    assert out[:, 0].isnan().all() and out[:, 65:].isnan().all() and out[15].isnan().all()


@pytest.mark.parametrize("dtype", TYPES)
def test_lookup_of_overlapping_rows(scr, dtype):
    """A table whose rows share memory gives what its copy gives; an output
    whose rows do is refused. Inside a larger buffer, so that a row taken from
    the wrong place is still a row of the buffer."""
    base = torch.randn(4096, generator=gen(30)).to(dtype).to(DEV)
    tok = torch.tensor([3, 0, -1, 6, 5, 7], device=DEV)
    for table in (base[:24].expand(7, 24), base[:40].unfold(0, 24, 1)[:7],
                  base[:200].unfold(0, 24, 8)[:7], base[5:29].expand(7, 24)):
        assert torch.equal(scr.embedding(tok, table, 0.5),
                           scr.embedding(tok, table.contiguous(), 0.5))
    table = base[:7 * 24].view(7, 24)
    one = torch.tensor([4], device=DEV)  # a single row may stand anywhere
    assert torch.equal(scr.embedding(one * 0, table[2:3].expand(1, 24)), table[2:3])
    out = torch.full((64, 24), 7.0, dtype=dtype, device=DEV)
    for bad in (out[:1].expand(6, 24), out.view(-1)[:64].unfold(0, 24, 8)[:6]):
        with pytest.raises(scr.CrError):
            scr.embedding(tok, table, out=bad)
    assert (out == 7).all()
    assert torch.equal(scr.embedding(one, table, out=out[:1].expand(1, 24))[0], table[4])


def tree(rows):
    """The canonical tree over rows (k, D) float32, column by column."""
    x = np.ascontiguousarray(rows.T.astype(np.float32))
    return oracle.reduce_batched(x.reshape(-1), x.shape[0], x.shape[1], 1, x.shape[1], 1,
                                 np.float32(-0.0))


def want_grad(tok, grad, V, scale):
    g = grad.float().numpy()
    out = np.zeros((V, g.shape[1]), np.float32)
    for v in range(V):
        at = np.nonzero(tok.numpy() == v)[0]
        if len(at):
            out[v] = tree(g[at]) * np.float32(scale)
    return out


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("n,V,D", [(1, 1, 1), (2, 3, 5), (700, 31, 77), (1037, 1500, 130),
                                   (5000, 3, 12), (4099, 300, 33), (0, 10, 16)])
def test_gradient_bits(scr, dtype, n, V, D):
    tok = skewed(n, V, 5)
    grad = torch.randn(n, D, generator=gen(6)).to(dtype)
    got = scr.embedding_backward(tok.to(DEV), grad.to(DEV), V, 0.3)
    assert got.dtype == torch.float32
    assert got.cpu().numpy().tobytes() == want_grad(tok, grad, V, 0.3).tobytes()


@pytest.mark.parametrize("count", [1, 7, 8, 9, 63, 64, 65, 127, 128, 200, 1000, 4096, 12345])
def test_gradient_of_one_frequent_token(scr, count):
    """Rows of every length around the sizes at which the tree is split."""
    n, V, D = count + 50, 20, 9
    tok = torch.randint(0, V, (n,), generator=gen(7))
    tok[torch.randperm(n, generator=gen(8))[:count]] = 11
    grad = torch.randn(n, D, generator=gen(9))
    got = scr.embedding_backward(tok.to(DEV), grad.to(DEV), V, 1.0)
    assert got.cpu().numpy().tobytes() == want_grad(tok, grad, V, 1.0).tobytes()


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("n,V,D,count", [(5000, 40, 1030, 3000), (700, 9, 520, 577),
                                         (9000, 700, 260, 8200), (17000, 300, 130, 15001)])
def test_gradient_of_long_rows(scr, dtype, n, V, D, count):
    """Long rows of many columns beside short ones: several warps to a row."""
    tok = torch.randint(0, V, (n,), generator=gen(22))
    tok[torch.randperm(n, generator=gen(23))[:count]] = 3
    grad = torch.randn(n, D, generator=gen(24)).to(dtype)
    got = scr.embedding_backward(tok.to(DEV), grad.to(DEV), V, 0.5)
    assert got.cpu().numpy().tobytes() == want_grad(tok, grad, V, 0.5).tobytes()


def test_gradient_large_vocabulary(scr):
    """More rows than one block sorts, and tokens of 32 bits."""
    n, V, D = 3000, 200_003, 4
    tok = skewed(n, V, 10)
    grad = torch.randn(n, D, generator=gen(11))
    got = scr.embedding_backward(tok.to(torch.int32).to(DEV), grad.to(DEV), V).cpu().numpy()
    used = np.unique(tok.numpy()[(tok.numpy() >= 0) & (tok.numpy() < V)])
    for v in used[::17]:
        assert got[v].tobytes() == tree(grad.numpy()[tok.numpy() == v]).tobytes()
    mask = np.ones(V, bool)
    mask[used] = False
    assert not got[mask].any()


@pytest.mark.parametrize("n", [1500, 6000])
def test_gradient_past_32_bits(scr, n):
    """Rows of the gradient that begin more than 2^31 elements into it."""
    V, D = (1 << 20) + 5000, 2052
    tok = torch.randint(V - 300, V, (n,), generator=gen(31))
    tok[:20] = torch.arange(20)
    grad = torch.randn(n, D, generator=gen(32)).to(torch.bfloat16)
    got = scr.embedding_backward(tok.to(DEV), grad.to(DEV), V, 0.5)
    assert got.numel() > 1 << 31
    assert not got[20:V - 300].any()
    want = want_grad(tok - (V - 300), grad, 300, 0.5)
    assert got[V - 300:].cpu().numpy().tobytes() == want.tobytes()
    assert torch.equal(got[:20].cpu(), grad[:20].float() * 0.5)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("n,V,D", [(500, 900, 68), (5000, 9000, 68), (3000, 2000, 37),
                                   (2048, 700, 130), (2049, 700, 130)])
def test_gradient_accumulates(scr, dtype, n, V, D):
    """out + scale * tree on rows with tokens, others untouched (NaN stays)."""
    tok = skewed(n, V, 12)
    grad = torch.randn(n, D, generator=gen(13)).to(dtype)
    old = torch.randn(V, D, generator=gen(14))
    have = np.isin(np.arange(V), tok.numpy())
    old[torch.from_numpy(~have)] = float("nan")
    out = old.to(DEV)
    r = scr.embedding_backward(tok.to(DEV), grad.to(DEV), V, 2.0, out=out, accumulate=True)
    assert r.data_ptr() == out.data_ptr()
    want = np.where(have[:, None], old.numpy() + want_grad(tok, grad, V, 2.0), old.numpy())
    assert out.cpu().numpy().tobytes() == want.astype(np.float32).tobytes()


def test_gradient_skips_padding_rows(scr):
    """Gradients of padding positions may hold anything."""
    tok = torch.tensor([3, -1, 5, 3, 99])
    grad = torch.randn(5, 40, generator=gen(15))
    grad[1], grad[4] = float("nan"), float("inf")
    got = scr.embedding_backward(tok.to(DEV), grad.to(DEV), 10).cpu()
    assert torch.equal(got[3], grad[0] + grad[3]) and torch.equal(got[5], grad[2])
    assert not got[[0, 1, 2, 4, 6, 7, 8, 9]].any()


@pytest.mark.parametrize("n", [200, 3000])
def test_gradient_strided(scr, n):
    tok = skewed(n, 30, 16)
    base = torch.full((n, 150), float("nan"))
    base[:, 5:138] = torch.randn(n, 133, generator=gen(17))
    out = torch.full((30, 140), -1.0, device=DEV)
    scr.embedding_backward(tok.to(DEV), base.to(DEV)[:, 5:138], 30, out=out[:, 3:136])
    got = out.cpu().numpy()
    assert got[:, 3:136].tobytes() == want_grad(tok, base[:, 5:138], 30, 1.0).tobytes()
    assert (got[:, :3] == -1).all() and (got[:, 136:] == -1).all()
    one = torch.randn(133, generator=gen(18))
    got = scr.embedding_backward(tok.to(DEV), one.to(DEV).expand(n, 133), 30).cpu().numpy()
    assert got.tobytes() == want_grad(tok, one.expand(n, 133), 30, 1.0).tobytes()


def test_gradient_matches_differences(scr):
    """The lookup is linear in its table: its change along a direction is the
    gradient's product with the direction."""
    tok = skewed(300, 40, 19)
    grad = torch.randn(300, 16, generator=gen(20))
    direction = torch.randn(40, 16, generator=gen(21))
    moved = scr.embedding(tok.to(DEV), direction.to(DEV), 0.7).cpu().double()
    dw = scr.embedding_backward(tok.to(DEV), grad.to(DEV), 40, 0.7).cpu().double()
    left, right = (moved * grad.double()).sum(), (dw * direction.double()).sum()
    # each side: 300 x 16 terms of one product, at most 300 roundings each
    scale = (moved * grad.double()).abs().sum()
    assert abs(left - right) <= 300 * 2.0 ** -23 * scale
