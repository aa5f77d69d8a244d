"""Four-bit attention at the ends of its ranges. Tolerances are test_kv4's unless a test says otherwise."""
import pytest

torch = pytest.importorskip("torch")
from test_kv4 import DT, _attend_case, on_gpu  # noqa: E402


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
