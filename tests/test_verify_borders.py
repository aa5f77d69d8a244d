"""The sampled selector and the verification beside the borders of their choices, with inputs whose borders
are known to far below a step of f32."""
import numpy as np
import pytest

from oracle import dflash_oracle as O

torch = pytest.importorskip("torch")
from test_verify import DT, _cu, on_gpu, sample_chain, softmax, verify  # noqa: E402


@pytest.fixture(scope="module", autouse=True)
def built():
    from speculative_block_drafter_gb300 import build
    build.build()


@on_gpu
@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("V,ld,top", [(37, None, 0), (5000, 5003, 0), (5000, 5003, 3), (50257, None, 2), (151936, None, 0)])
def test_verify_decides_beside_the_border(dtype, V, ld, top):
    """Uniform numbers one f32 step to either side of p / q, or on it: the draft is kept exactly below it,
    whatever the row's alignment. Rows whose border lies within 2^-38 / p of the number (relative: twice what
    the weights carry) are left out, which is no input that a test of f32 numbers would meet."""
    from speculative_block_drafter_gb300 import drafter as D
    rng = np.random.default_rng(V + top)
    b, k = (6, 9) if V > 100000 else (24, 9)
    x = rng.standard_normal((b, k + 1, V)).astype(np.float32)
    d = rng.integers(0, V, (b, k))
    T = np.where(np.arange(b) % 2 == 0, 1.0, 0.6 + 0.6 * rng.random(b)).astype(np.float32)
    share = np.log(0.1 + 0.5 * rng.random((b, k)))             # of the draft against all others, about
    hot = T[:, None] * (np.log(V) + 0.5 / T[:, None] ** 2 + share)
    np.put_along_axis(x[:, :k], d[:, :, None], hot[:, :, None].astype(np.float32), 2)
    x = torch.from_numpy(x).to(DT[dtype])
    cand = q = None
    if top:
        cand = (d[:, :, None] + np.arange(top)) % V            # the draft itself first
        q = (0.85 + 0.1 * rng.random((b, k, top))).astype(np.float32)
    xf = x.float().numpy()
    u = np.zeros((b, k + 1), np.float32)
    u[:, k] = rng.random(b)
    for i in range(b):
        for j in range(k):
            w = softmax(xf[i, j], float(T[i]))
            p, qj = w[d[i, j]] / w.sum(), float(q[i, j, 0]) if top else 1.0
            r = np.float32(p / qj)
            assert 0 < r < 0.999
            # the largest number below the border; for the row's last draft the smallest that is not below it
            r = r if float(r) * qj < p else np.nextafter(r, np.float32(0))
            if (i + j) % 5 == 4:
                r = np.nextafter(r, np.float32(1))
            if abs(float(r) * qj - p) < 2.0 ** -38:
                r = np.float32(0.5) * r
            u[i, j] = r
    wide = x.cuda()
    if ld is not None:                                         # rows further apart, from an odd address
        wide = torch.full((b * (k + 1) * ld + 1,), float("nan"), dtype=x.dtype, device="cuda")[1:].view(b, k + 1, ld)
        wide = wide[:, :, :V]
        wide.copy_(x)
    acc, tok = D.verify(wide, _cu(d, torch.int32), _cu(u), temperature=_cu(T), cand=_cu(cand, torch.int32) if top else None,
                        cand_q=_cu(q) if top else None)
    acc, tok = acc.cpu().numpy(), tok.cpu().numpy()
    for i in range(b):
        # (f64 uniforms: an f32 one times a probability would be rounded to f32)
        ref = verify(xf[i], d[i], u[i].astype(np.float64), float(T[i]), cand[i] if top else None, q[i] if top else None, k)
        assert (acc[i], list(tok[i])) == ref, i
    assert 0 < acc.sum() < b * k


@on_gpu
@pytest.mark.parametrize("rank,top", [(16, 8), (64, 16), (256, 32)])
def test_select_sample_keeps_what_f32_scores_would_lose(rank, top):
    """Candidates whose scores agree to an f32 step, at a temperature of a few such steps: the probabilities
    turn on parts of the products below f32. The low part of a sum of n terms takes up n errors of 2^-24 of
    the terms' sizes together, and adding those up in f32 costs another 2^-24 of it each time: n^2 2^-48 in all.
    Over the temperature that is the weights' relative error, twice (the weight and the largest one), to which
    the probabilities' own (2^-24, 2^-39) come."""
    from speculative_block_drafter_gb300 import drafter as D
    rng = np.random.default_rng(rank)
    V, b = 512, 48
    pred, succ = ((rng.standard_normal((V, rank)) / rank ** 0.25).astype(np.float16) for _ in range(2))
    hp = rng.standard_normal((b, 1, rank)).astype(np.float32)
    anchor = rng.integers(0, V, b)
    logits = np.full((b, 1, V), -200.0, np.float32)
    size = np.zeros(b)
    for i in range(b):
        a = pred[anchor[i]].astype(np.float64) * hp[i, 0].astype(np.float64)
        cand = rng.permutation(V)[:top]
        logits[i, 0, cand] = (6.0 - succ[cand].astype(np.float64) @ a).astype(np.float32)
        size[i] = (np.abs(succ[cand].astype(np.float64)) @ np.abs(a) + np.abs(logits[i, 0, cand])).max()
    T = np.full(b, 2.0 ** -21, np.float32)
    u = rng.random((b, 1)).astype(np.float32)
    _, cand, q = D.select_sample(_cu(logits), _cu(hp), _cu(anchor, torch.int32), _cu(pred), _cu(succ), top, _cu(T), _cu(u))
    cand, q = cand.cpu().numpy(), q.cpu().numpy().astype(np.float64)
    spread = 0
    for i in range(b):
        _, rcand, rq = sample_chain(logits[i], hp[i], int(anchor[i]), pred, succ, top, float(T[i]), u[i])
        assert np.array_equal(cand[i], rcand)
        tol = (2.0 ** -24 + 2 * rank ** 2 * 2.0 ** -48 * size[i] / T[i]) * rq + 2.0 ** -39
        assert np.all(np.abs(q[i] - rq) <= tol), float((np.abs(q[i] - rq) / tol).max())
        spread += (rq > 0.02).sum() > 1
    assert spread > b / 2                                      # near ties, as they are meant to be


@on_gpu
@pytest.mark.parametrize("zeros", [1, 30, 3000])
def test_selectors_take_the_two_zeros_as_equal(zeros):
    """Rows whose largest logits are zeros of both signs: equal values, so the lower index first, within a chunk
    of the rows, across chunks and past what a candidate list holds."""
    from speculative_block_drafter_gb300 import _lib as L
    from speculative_block_drafter_gb300 import drafter as D
    rng = np.random.default_rng(zeros)
    b, k, V, rank, top = 3, 5, 5000, 16, 8
    logits = -1 - rng.random((b, k, V)).astype(np.float32)
    for row in logits.reshape(-1, V):
        row[rng.permutation(V)[:zeros]] = np.where(rng.random(zeros) < 0.5, 0.0, -0.0)
    pred, succ = ((rng.standard_normal((V, rank)) / 4).astype(np.float16) for _ in range(2))
    hp = rng.standard_normal((b, k, rank)).astype(np.float32)
    anchor = rng.integers(0, V, b)
    u = rng.random((b, k)).astype(np.float32)
    t = [_cu(logits), _cu(hp), _cu(anchor, torch.int32), _cu(pred), _cu(succ)]
    ch, cand, _ = D.select_sample(*t, top, None, _cu(u))
    best, plain = (torch.empty(b, k, dtype=torch.int32, device="cuda") for _ in range(2))
    L.dflash_select_static(*(x.data_ptr() for x in t), b, k, V, V, rank, top, best.data_ptr(), plain.data_ptr(),
                           torch.cuda.current_stream().cuda_stream)
    for i in range(b):
        rc, rcand, _ = sample_chain(logits[i], hp[i], int(anchor[i]), pred, succ, top, 1.0, u[i])
        assert np.array_equal(cand[i].cpu().numpy(), rcand) and list(ch[i].cpu().numpy()) == list(rc)
        chosen, first = O.select_with(hp[i], logits[i], int(anchor[i]), pred, succ, top)
        assert list(best[i].cpu().numpy()) == list(chosen) and list(plain[i].cpu().numpy()) == list(first)
