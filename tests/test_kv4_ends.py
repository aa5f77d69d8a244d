"""Four-bit attention at the ends of its ranges. Tolerances are test_kv4's unless a test says otherwise."""
import pytest

torch = pytest.importorskip("torch")
from test_kv4 import DT, _attend_case, _cache, on_gpu, quantise  # noqa: E402


@pytest.fixture(scope="module", autouse=True)
def built():
    from speculative_block_drafter_gb300 import build
    build.build()


@on_gpu
@pytest.mark.parametrize("dtype,hd,R,heads,kv", [("f32", 64, 4, 2, 1), ("f32", 128, 3, 4, 2), ("f32", 128, 16, 4, 1),
                                                 ("f32", 64, 16, 2, 1), ("bf16", 64, 4, 2, 1)])
@pytest.mark.parametrize("window,causal", [(0, False), (40, True)])
def test_attention_of_subnormal_query_rows(dtype, hd, R, heads, kv, window, causal):
    """Query rows whose largest value is subnormal, or small enough for the factor from products to scores to
    leave f32's range, beside ordinary ones, over a range that ends inside a group of 16 rows: scores of 0 in
    effect, so the mean of the values seen."""
    g = torch.Generator().manual_seed(hd + R)
    q = torch.randn(1, R, heads, hd, generator=g)
    q[0, 0] *= 1e-44
    q[0, 1] = 2.0 ** -140
    q[0, 2] *= 1e-38
    _attend_case(dtype, 1, R, heads, kv, hd, 300, [0], [300], [290], window, causal, q=q.to(DT[dtype]))
    _attend_case(dtype, 1, R, heads, kv, hd, 300, [0], [300], [290], window, causal,
                 q=torch.randn(1, R, heads, hd, generator=g).to(DT[dtype]), scale=1e-42)


@on_gpu
@pytest.mark.parametrize("dtype,hd,R,heads,kv", [("f32", 64, 4, 2, 1), ("f32", 128, 2, 4, 1), ("bf16", 128, 1, 8, 2),
                                                 ("f32", 64, 64, 2, 2), ("f32", 128, 32, 2, 2), ("bf16", 128, 60, 2, 2)])
@pytest.mark.parametrize("sign", [-1, 1])
def test_attention_of_scores_of_any_size(dtype, hd, R, heads, kv, sign):
    """Scores from 1e3 to beyond 1e31, of either sign, one key's at least three times the distance from 0 of
    every other (or a quarter of it, below 0): all weight is on that key, whatever f32 keeps of the scores, and
    the output is its value. Ranges that some queries see only from their second tile on."""
    g = torch.Generator().manual_seed(R)
    n, at, lo, window = 700, 690, 100, 700 - 100
    k = torch.full((1, n, kv, hd), sign * (0.4375 if sign > 0 else 1.75))
    k[:, at] = sign * (1.75 if sign > 0 else 0.4375)
    v = torch.randn(1, n, kv, hd, generator=g)
    mag = torch.logspace(3, 31, R * heads).view(R, heads)
    mag = mag[torch.randperm(R, generator=g)]
    q = (mag.unsqueeze(-1) * (hd ** -0.5)).expand(1, R, heads, hd).to(DT[dtype])
    c = _cache(1, n, kv, hd)
    c.write([0], k.cuda(), v.cuda())
    want = quantise(v)[0, at].float().repeat_interleave(heads // kv, 0).to(DT[dtype])
    for a in (dict(window=0), dict(window=window, causal=True)):
        # with the window, query r sees the rows from lo + r on
        y, lse = c.attend(q.cuda(), [lo], [n], [n - 1], lse=True, **a)
        y, lse = y.cpu().double(), lse.cpu().double()
        # one weight against itself: its two planes and the sum, 2^-22 each, and the output's rounding
        assert bool(((y[0] - want.double()).abs() <= (2.0 ** -20 + (2.0 ** -7 if dtype != "f32" else 0)) * want.double().abs()).all())
        s = q[0].double().sum(-1) * hd ** -0.5 * float(k[0, at, 0, 0])
        assert bool(((lse[0] - s).abs() <= (hd + 8) * 2.0 ** -22 * s.abs()).all())


@on_gpu
@pytest.mark.parametrize("dtype,hd,R,heads", [("f32", 64, 4, 2), ("f32", 128, 32, 2), ("f16", 128, 1, 8)])
def test_attention_of_large_random_scores_stays_among_the_values(dtype, hd, R, heads):
    """Random scores of 1e2 to 1e33, which f32 keeps to their leading bits only: the output is finite and a
    mean of values (2^-10 for the weights' rounding and the sums, and the output's rounding)."""
    g = torch.Generator().manual_seed(R)
    n = 900
    mag = torch.logspace(2, 33 if dtype != "f16" else 4, R * heads).view(R, heads, 1)
    q = (torch.randn(R, heads, hd, generator=g) * mag).unsqueeze(0).to(DT[dtype])
    k, v = (torch.randn(1, n, 1, hd, generator=g) for _ in range(2))
    c = _cache(1, n, 1, hd)
    c.write([0], k.cuda(), v.cuda())
    held = quantise(v)[0, :, 0]
    top = held.abs().amax(0) * (1 + 2.0 ** -6)
    for causal in (False, True):
        y, lse = c.attend(q.cuda(), [0], [n], [n - 40], causal=causal, lse=True)
        y = y.cpu().double()[0]
        assert bool(torch.isfinite(y).all()) and bool(torch.isfinite(lse).all())
        assert bool((y.abs() <= top).all())
        # no row's weights have vanished: a mean of values of +-1 and more is not 0 everywhere
        assert bool((y.abs().amax(-1) > 0).all())
