"""Four-bit attention at the ends of its ranges. Tolerances are test_kv4's unless a test says otherwise."""
import pytest

torch = pytest.importorskip("torch")
from test_kv4 import DT, _attend_case, _cache, _lib, attend, on_gpu, quantise, tolerance  # noqa: E402


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


@on_gpu
@pytest.mark.parametrize("dtype,hd,R,rep,n", [("f32", 128, 16, 2, 1 << 17), ("f32", 128, 32, 2, 1 << 17), ("f32", 64, 48, 1, 1 << 17),
                                              ("f16", 128, 16, 3, 1 << 19), ("f32", 64, 4, 2, 1 << 20), ("f32", 128, 16, 1, 1 << 19)])
@pytest.mark.parametrize("flat", [True, False])
def test_attention_sums_do_not_drift_over_many_rows(dtype, hd, R, rep, n, flat):
    """160 pairs of 131,072 rows and more, some CTA's piece as long: the error does not grow with the rows.
    A sum stays in the matrix instructions for 256 of their steps at most, each of which may cut off 2^-22 of
    it (2^-23 of the sum so far, as much of the products beside it): twice what the tolerance has a step for.
    Flat: equal scores and values. Else: scores that swing by 40 along the rows, so that the references move
    within the runs and between them."""
    kv = 160
    g = torch.Generator().manual_seed(R)
    k, v = torch.zeros(1, n, 1, hd), torch.full((1, n, 1, hd), 1.75)
    q = torch.randn(1, R, rep, hd, generator=g)
    if not flat:
        at = torch.arange(n) * (2 * 3.14159 / 50000)
        k[0, :, 0, 0], k[0, :, 0, 1] = at.sin(), at.cos()
        phase = torch.rand(R, rep, generator=g) * 6.28
        q[0, :, :, 0], q[0, :, :, 1] = 20 * hd ** 0.5 * phase.cos(), 20 * hd ** 0.5 * phase.sin()
        v = torch.randn(1, n, 1, hd, generator=g) + 1
    q = q.to(DT[dtype])
    one = _cache(1, n, 1, hd)
    one.write([0], k.cuda(), v.cuda())
    c = _cache(1, n, kv, hd)
    c.k.copy_(one.k.expand_as(c.k))
    c.v.copy_(one.v.expand_as(c.v))
    y = c.attend(q.unsqueeze(2).expand(1, R, kv, rep, hd).reshape(1, R, kv * rep, hd).cuda(), [0], [n], [n])
    hk, hv = (t[:, 0].cuda().double() for t in (quantise(k)[0], quantise(v)[0]))
    p = torch.softmax(torch.einsum("rhd,nd->rhn", q[0].cuda().double(), hk) * hd ** -0.5, -1)
    want, bound = p @ hv, (p @ hv.abs()).amax(-1)
    tol = tolerance(dtype, hd, 2 * 16 * 256, bound.cpu(), want.cpu()).cuda()
    err = (y.view(R, kv, rep, hd).double() - want.unsqueeze(1)).abs().amax(-1)
    assert bool((err <= tol.unsqueeze(1)).all()), float((err / tol.unsqueeze(1)).max())


@on_gpu
@pytest.mark.parametrize("dtype,hd,R,rep", [("f32", 128, 32, 2), ("f32", 128, 16, 2), ("f32", 64, 2, 1), ("f16", 64, 9, 4)])
def test_attention_of_long_and_short_pairs_together(dtype, hd, R, rep):
    """480 pairs of 100,000, 333, none and 20,000 rows, all from inside a tile, so that a CTA's pieces are of
    one run or several, whole and divided, one after another; causal, and the same bits every time."""
    kv, lo, hi = 120, [5, 1000, 40, 129], [100005, 1333, 40, 20129]
    g = torch.Generator().manual_seed(hd + R)
    n = max(hi)
    k, v = (torch.randn(4, n, 1, hd, generator=g) for _ in range(2))
    q = torch.randn(4, R, rep, hd, generator=g).to(DT[dtype])
    one = _cache(4, n, 1, hd)
    one.write([0] * 4, k.cuda(), v.cuda())
    c = _cache(4, n, kv, hd)
    c.k.copy_(one.k.expand_as(c.k))
    c.v.copy_(one.v.expand_as(c.v))
    args = (q.unsqueeze(2).expand(4, R, kv, rep, hd).reshape(4, R, kv * rep, hd).cuda(), lo, hi, [x - R for x in hi])
    args[3][2] = 0
    y, lse = c.attend(*args, causal=True, lse=True)
    y2 = c.attend(*args, causal=True)
    assert torch.equal(y, y2)
    y, lse = y.view(4, R, kv, rep, hd).cpu().double(), lse.view(4, R, kv, rep).cpu().double()
    for b in range(4):
        ry, rl, bound = attend(q[b], quantise(k[b]), quantise(v[b]), lo[b], hi[b], args[3][b], 0, True, hd ** -0.5)
        tol = tolerance(dtype, hd, min(hi[b] - lo[b], 2 * 16 * 256), bound, ry)
        assert bool(((y[b] - ry.unsqueeze(1)).abs().amax(-1) <= tol.unsqueeze(1)).all()), b
        if hi[b] > lo[b]:
            # a thread adds up at most 256 weights of a run, and the runs are joined in f32
            assert bool(((lse[b] - rl.unsqueeze(1)).abs() <= (hd + 8 + 300) * 2.0 ** -22 + 2.0 ** -22 * rl.abs().max()).all())
        else:
            assert bool((lse[b] == float("-inf")).all()) and bool((y[b] == 0).all())


@on_gpu
@pytest.mark.parametrize("dtype,hd,R,rep", [("f32", 128, 4, 1), ("f32", 128, 16, 1), ("f32", 64, 16, 2), ("f32", 128, 16, 2),
                                            ("f32", 128, 32, 2), ("f32", 64, 48, 1), ("bf16", 128, 1, 4), ("f16", 128, 16, 2),
                                            ("bf16", 64, 16, 4)])
@pytest.mark.parametrize("spike", [0, 16500])
def test_attention_keeps_a_long_tail_under_one_large_weight(dtype, hd, R, rep, spike):
    """One row 12 to 24 nats above 32,768 equal ones, whose values alone are not 0: the output is the tail's
    share. A weight enters the products to 2^-34 of the largest of its run at worst, and a run has at most
    8,192 rows, so beside the tolerance the output may be off by 2^-34 of the value for each of those. 320
    pairs, so that a CTA has a pair or more and full runs meet the one row's reference."""
    n, kv, batch, V = 32769, 160, 2, 1.75                      # 7 * 0.25: held exactly
    k, v = torch.zeros(1, n, 1, hd), torch.full((1, n, 1, hd), V)
    k[0, spike] = V
    v[0, spike] = 0
    one = _cache(1, n, 1, hd)
    one.write([0], k.cuda(), v.cuda())
    c = _cache(batch, n, kv, hd)
    c.k.copy_(one.k.expand_as(c.k))
    c.v.copy_(one.v.expand_as(c.v))
    gap = torch.linspace(12, 24, R * rep).view(R, 1, rep, 1)
    q = (gap / (V * hd ** 0.5)).expand(R, kv, rep, hd).reshape(1, R, kv * rep, hd).expand(batch, -1, -1, -1).to(DT[dtype])
    y = c.attend(q.cuda(), [0] * batch, [n] * batch, [n] * batch).cpu().double()
    s = q[0, :, :rep].double().sum(-1) * V * hd ** -0.5         # the large score; the others are 0
    w = (n - 1) * torch.exp(-s)
    want = (V * w / (1 + w)).view(1, R, 1, rep, 1)
    tol = tolerance(dtype, hd, n, want[..., 0], want) + 8192 * 2.0 ** -34 * V
    err = (y.view(batch, R, kv, rep, hd) - want).abs().amax(-1)
    assert bool((err <= tol).all()), float((err / tol).max())


@on_gpu
@pytest.mark.parametrize("dtype,R", [("f32", 17), ("bf16", 48)])
def test_attention_of_pairs_that_see_nothing_between_others(dtype, R):
    """2,560 pairs of one tile each, a CTA's many pieces taking turns between ranges that are empty, seen by the
    last query rows only, and full: every query's reference starts over with its piece."""
    hi = [(0, 100, 128)[b % 3] for b in range(64)]
    anchor = [(0, 128, 127)[b % 3] for b in range(64)]
    lo = [(0, 60, 0)[b % 3] for b in range(64)]
    y = _attend_case(dtype, 64, R, 40, 40, 128, 128, lo, hi, anchor, window=40 + R)
    assert bool((y[0] == 0).all()) and bool((y[2] != 0).any())


@on_gpu
@pytest.mark.parametrize("R", [1, 40])
def test_attention_over_the_longest_cache(R):
    """A cache of 2^31 - 1 rows, whose last tile's last row is not one of them: all rows alike, at a score of
    about -100, so that a row read past the end (a score of 0) would take all the weight. K and V are one buffer
    of 77 GB."""
    L = _lib()
    rows, hd = (1 << 31) - 1, 64
    if torch.cuda.mem_get_info()[0] < 100 << 30:
        pytest.skip("needs 100 GB of device memory")
    nb = L.dflash_kv4_cache_bytes(1, hd, rows)
    from speculative_block_drafter_gb300.drafter import kv4_values
    c = torch.full((nb,), 0x18, dtype=torch.uint8, device="cuda")     # codes of 0 and -7, scales of eight bits
    x = kv4_values(c[:128 * (hd // 2 + hd // 16)].view(1, -1), hd)[0]
    q = torch.full((1, R, 1, hd), -100 * hd ** 0.5 / float(x.sum()), device="cuda")
    y, lse = torch.empty_like(q), torch.empty(1, R, 1, device="cuda")
    wb = L.dflash_kv4_attention_workspace_bytes(1, R, 1, 1, hd)
    ws = torch.empty(wb, dtype=torch.uint8, device="cuda")
    L.dflash_kv4_attention(1, R, 1, 1, hd, rows, L.pointers([c.data_ptr()]), L.pointers([c.data_ptr()]), L.int64s([0]),
                           L.int64s([rows]), L.int64s([rows]), 0, 0, hd ** -0.5, q.data_ptr(), R * hd, hd, 0,
                           y.data_ptr(), lse.data_ptr(), ws.data_ptr(), wb,
                           torch.cuda.current_stream().cuda_stream)
    torch.cuda.synchronize()
    del c
    torch.cuda.empty_cache()
    assert L.dflash_device_error(reset=True) == 0
    # a run's sums are off by 256 steps of 2^-22, joined in f32 in 3,449 runs of a CTA and 152 partials
    assert bool(((y - x).abs() <= (256 * 2.0 ** -22 + 3601 * 2.0 ** -24) * x.abs()).all())
    assert bool((lse - (torch.log(torch.tensor(float(rows))).item() - 100)).abs().max() < 1e-3)
