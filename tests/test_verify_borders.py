"""The sampled selector and the verification beside the borders of their choices, with inputs whose borders
are known to far below a step of f32."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")
from test_verify import DT, _cu, on_gpu, softmax, verify  # noqa: E402


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
