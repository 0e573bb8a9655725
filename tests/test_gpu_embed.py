"""The embedding lookup and its gradient by sorted tokens: both types and index
types, odd widths and strides, padded tokens, tokens that fill many pieces of the
sorted rows, vocabularies of one to three passes, adding into an array, far
offsets, capture, refusals.  The lookup is one rounded product (and another rounding
for bf16: 2^-24 of the value); the gradient's bound is lm_ref.py's."""
import pytest
import torch

from tests import lm_ref as L
from tests import ssm_ref as R

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32
I32, I64 = torch.int32, torch.int64


@pytest.fixture(scope="module")
def g():
    from linear_attention_sequence_device_gb300 import build
    build.build_library()
    import linear_attention_sequence_device_gb300 as pkg
    pkg.load()
    return pkg


@pytest.fixture(autouse=True)
def memory():
    yield
    torch.cuda.empty_cache()


def gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def view(T, W, dtype, q, pad=0, skip=0):
    """[T, W] with row stride W + pad, `skip` elements behind an aligned address."""
    flat = torch.randn(T * (W + pad) + skip, generator=q, device="cuda").to(dtype)
    return flat[skip:].view(T, W + pad)[:, :W]


SHAPES = [(1, 1, 1, BF, I64), (7, 3, 5, F32, I32), (300, 50, 64, BF, I32), (1000, 2000, 4096, BF, I64), (513, 40, 2056, F32, I64),
          (4096, 9, 33, BF, I64), (4097, 70000, 40, F32, I32), (0, 5, 8, BF, I64), (64, 1 << 18, 8, BF, I64)]


@pytest.mark.parametrize("T,V,W,dtype,index", SHAPES)
@pytest.mark.parametrize("pad,skip", [(0, 0), (8, 0), (3, 1)])
def test_lookup(g, T, V, W, dtype, index, pad, skip):
    q = gen(0)
    table = view(V, W, dtype, q, pad, skip)
    tok = torch.randint(-2, V + 2, (T,), generator=q, device="cuda").to(index)
    real = (tok >= 0) & (tok < V)
    ref = torch.where(real[:, None], L.dbl(table)[tok.long().clamp(0, V - 1)], 0.0)
    for scale in (1.0, -2.7):
        y = g.gdn_embed_fwd(tok, table, scale=scale)
        # the scale is an fp32 number: -2.7 is rounded by up to U of itself before any product
        most = L.U * (ref * scale).abs() * (1.01 * (dtype is BF) + (scale != 1.0))
        R.assert_within(y, (ref * scale).cpu(), most.cpu() + 1e-300, "y")
    out = view(T, W, dtype, q, 5)
    assert g.gdn_embed_fwd(tok, table, out=out) is out and torch.equal(out, g.gdn_embed_fwd(tok, table))


def tokens(kind, T, V, q):
    if kind == "one":
        return torch.full((T,), V - 1, device="cuda")
    if kind == "padded":
        return torch.full((T,), -1, device="cuda")
    if kind == "runs":  # every length of a run around the pieces' 16 rows
        n = torch.arange(1, 2 * T, device="cuda")
        return torch.repeat_interleave(n, n % 70)[:T][torch.randperm(T, generator=q, device="cuda")] % V
    r = torch.rand(T, generator=q, device="cuda").double()
    t = torch.exp(r * torch.log(torch.tensor(V + 1.0, device="cuda").double())).long() - 1  # the long tail of text
    t[torch.rand(T, generator=q, device="cuda") < 0.1] = -1
    t[torch.rand(T, generator=q, device="cuda") < 0.05] = V + 7
    return t


GRAD = [("tail", 1, 1, 1, BF, I64), ("tail", 7, 3, 5, F32, I32), ("tail", 300, 50, 64, BF, I32), ("runs", 3000, 400, 72, BF, I64),
        ("runs", 4096, 40, 1100, F32, I64), ("runs", 20000, 3000, 40, F32, I32), ("one", 5000, 3, 2056, BF, I64),
        ("one", 16, 2, 8, F32, I64), ("one", 33, 2, 8, F32, I64), ("padded", 100, 5, 24, BF, I64), ("padded", 9000, 5, 24, F32, I32),
        ("tail", 40000, 70000, 264, BF, I64), ("tail", 4097, 1 << 19, 8, F32, I64), ("tail", 70000, 9, 17, F32, I64),
        ("tail", 0, 6, 8, BF, I64), ("runs", 2049 * 16, 500, 16, BF, I32)]


@pytest.mark.parametrize("kind,T,V,W,dtype,index", GRAD)
def test_gradient(g, kind, T, V, W, dtype, index):
    q = gen(1)
    tok = tokens(kind, T, V, q).to(index)
    for pad, skip, scale in ((0, 0, 1.0), (8, 0, 1.5), (3, 1, -0.3)):
        dy = view(T, W, dtype, q, pad, skip)
        d = g.gdn_embed_bwd(dy, tok, V, scale=scale)
        ref, bound = L.embed_bwd(L.dbl(dy), tok.long(), V, scale)
        R.assert_within(d, ref.cpu(), (bound + 2 * L.U * ref.abs()).cpu(), "dtable")
        assert torch.equal(d, g.gdn_embed_bwd(dy, tok, V, scale=scale))  # equal calls, equal bits


@pytest.mark.parametrize("kind,T,V,W,dtype,index", [c for c in GRAD if c[1] in (300, 3000, 5000, 100, 0, 4097)])
def test_gradient_into_another(g, kind, T, V, W, dtype, index):
    """The rows of tokens that occur are added to; no other row is touched, nor what lies between two rows."""
    q = gen(2)
    tok, dy = tokens(kind, T, V, q).to(index), view(T, W, dtype, q)
    whole = torch.randn(V, W + 8, generator=q, device="cuda").to(dtype)
    old = whole.clone()
    d = g.gdn_embed_bwd(dy, tok, V, scale=0.5, into=whole[:, :W])
    ref, bound = L.embed_bwd(L.dbl(dy), tok.long(), V, 0.5)
    R.assert_within(d, (L.dbl(old[:, :W]) + ref).cpu(), (bound + 2 * L.U * (ref.abs() + L.dbl(old[:, :W]).abs())).cpu(), "into")
    hit = torch.zeros(V, dtype=torch.bool, device="cuda")
    hit[tok[(tok >= 0) & (tok < V)].long()] = True
    assert torch.equal(whole[~hit], old[~hit]) and torch.equal(whole[:, W:], old[:, W:])


def test_rows_do_not_leak(g):
    """Padded tokens' gradients are not read; NaN reaches the rows of its token alone."""
    q = gen(3)
    tok = torch.randint(0, 40, (500,), generator=q, device="cuda")
    dy = view(500, 64, F32, q)
    tok[::7] = -1
    clean = g.gdn_embed_bwd(dy, tok, 40)
    dy[::7] = float("nan")
    dy[1] = float("inf")
    d = g.gdn_embed_bwd(dy, tok, 40)
    keep = torch.arange(40, device="cuda") != tok[1]
    assert torch.equal(d[keep], clean[keep]) and not torch.isfinite(d[tok[1]]).any()


def test_a_longer_calls_workspace(g):
    q = gen(4)
    ws = torch.full((g.embed_bwd_workspace_size(9000, 30, 64),), 255, dtype=torch.uint8, device="cuda")
    sizes = [g.embed_bwd_workspace_size(T, 30, 64) for T in (0, 1, 4096, 4097, 32768, 32769, 70000, 600000, 1 << 22)]
    assert sizes == sorted(sizes)
    for T in (1, 100, 5000, 9000):
        dy, tok = view(T, 64, BF, q), torch.randint(0, 30, (T,), generator=q, device="cuda")
        assert torch.equal(g.gdn_embed_bwd(dy, tok, 30, workspace=ws), g.gdn_embed_bwd(dy, tok, 30))


def test_far_rows(g):
    """Rows of the table and of its gradient beyond 2^31 elements."""
    W, V = 4096, 2 ** 31 // 4096 + 100
    q = gen(5)
    table = torch.empty(V, W, dtype=BF, device="cuda")
    table[-64:] = torch.randn(64, W, generator=q, device="cuda").to(BF)
    tok = V - 1 - torch.randint(0, 64, (50,), generator=q, device="cuda")
    assert torch.equal(g.gdn_embed_fwd(tok, table), table[tok])
    dy = view(50, W, BF, q)
    d = g.gdn_embed_bwd(dy, tok, V)
    near = g.gdn_embed_bwd(dy, tok - (V - 64), 64)
    assert torch.equal(d[-64:], near) and not d[:64].any() and not d[-200:-64].any()


def test_far_tokens(g):
    """Rows of the result and of dy beyond 2^31 elements."""
    W, T = 4096, 2 ** 31 // 4096 + 77
    q = gen(6)
    table = torch.randn(9, W, generator=q, device="cuda").to(BF)
    tok = torch.randint(0, 9, (T,), generator=q, device="cuda")
    y = g.gdn_embed_fwd(tok, table)
    assert torch.equal(y[-300:], table[tok[-300:]])
    tok[:-300] = -1
    assert torch.equal(g.gdn_embed_bwd(y, tok, 9), g.gdn_embed_bwd(y[-300:], tok[-300:], 9))


def test_captured_on_another_stream(g):
    q = gen(7)
    dy, tok, table = view(6000, 64, BF, q), torch.randint(0, 3000, (6000,), generator=q, device="cuda"), view(3000, 64, BF, q)
    dy2, tok2 = view(6000, 64, BF, q), torch.randint(-1, 3000, (6000,), generator=q, device="cuda") // 300
    both = lambda: (g.gdn_embed_fwd(tok, table), g.gdn_embed_bwd(dy, tok, 3000))
    want = g.gdn_embed_fwd(tok2, table), g.gdn_embed_bwd(dy2, tok2, 3000)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        both()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = both()
    dy.copy_(dy2)
    tok.copy_(tok2)
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))


def test_gradient_against_differences(g):
    """<dy, y(table + s D) - y(table - s D)> / 2s is <dtable, D>: the lookup is linear, so only rounding counts."""
    q = gen(8)
    table, D = torch.randn(2, 20, 16, generator=q, device="cuda")
    tok, dy = torch.randint(-1, 20, (200,), generator=q, device="cuda"), view(200, 16, F32, q)
    diff = L.dbl(g.gdn_embed_fwd(tok, table + D, scale=3.0)) - L.dbl(g.gdn_embed_fwd(tok, table - D, scale=3.0))
    left = float((L.dbl(dy) * diff).sum() / 2)
    right = float((L.dbl(g.gdn_embed_bwd(dy, tok, 20, scale=3.0)) * L.dbl(D)).sum())
    # 3200 products, each off by a few roundings of terms of order ten
    assert abs(left - right) <= 3200 * 16 * L.U * 10


def test_wrong_arguments_raise(g):
    q = gen(9)
    table, tok, dy = view(9, 16, BF, q), torch.zeros(5, dtype=I64, device="cuda"), view(5, 16, BF, q)
    with pytest.raises(TypeError):
        g.gdn_embed_fwd(tok.float(), table)
    with pytest.raises(ValueError):
        g.gdn_embed_fwd(tok.cpu(), table)
    with pytest.raises(ValueError):
        g.gdn_embed_fwd(tok[:, None], table)
    with pytest.raises(ValueError):
        g.gdn_embed_fwd(tok, table, out=dy[:4])
    with pytest.raises(ValueError):
        g.gdn_embed_fwd(tok, table.t())
    with pytest.raises(ValueError):
        g.gdn_embed_bwd(dy, tok[:4], 9)
    with pytest.raises(TypeError):
        g.gdn_embed_bwd(dy, tok, 9, into=torch.zeros(9, 16, device="cuda"))
    with pytest.raises(g.GdnError):
        g.gdn_embed_bwd(dy, tok, 9, workspace=torch.empty(256, dtype=torch.uint8, device="cuda"))
    with pytest.raises(TypeError):
        g.gdn_embed_fwd(tok, table.half())
