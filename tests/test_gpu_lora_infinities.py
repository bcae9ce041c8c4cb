"""Infinities in x, in an adapter and in its sums, in tiles of few rows and of 128: the outputs that the formula makes infinite
are, those that it makes NaN are NaN, and the others are what they were."""
import pytest
import torch

import linear_ref as ref

pytestmark = pytest.mark.gpu

BF16, F16 = torch.bfloat16, torch.float16
SIZES = [(1, 1, 8, 64, 48), (40, 3, 24, 512, 96), (100, 2, 128, 1024, 320), (9000, 2, 72, 2560, 496), (20000, 2, 32, 2048, 1024)]


def data(T, G, r, H, N, dtype):
    g = torch.Generator(device="cuda").manual_seed(T)
    normal = lambda *shape, scale=1.0: (torch.randn(*shape, generator=g, device="cuda") * scale).to(dtype)
    ids = torch.randint(0, G, (T, 1), generator=g, device="cuda", dtype=torch.int32)
    # no zeros, so that an infinity's products are infinite
    nonzero = lambda t: torch.where(t == 0, torch.ones_like(t), t)
    return ids, normal(T, N), nonzero(normal(T, H)), nonzero(normal(G, r, H, scale=H ** -0.5)), nonzero(normal(G, N, r, scale=r ** -0.5))


def check(ids, y, x, a, b):
    import combine_topk_ids_histogram_gb300 as ep
    L = ep.dispatch_layout(ids, a.shape[0])
    out = ep.lora_add(y, x, a, b, L)
    assert ep.read_status(L) == 0
    want, tol = y.double(), torch.zeros(y.shape, dtype=torch.float64, device="cuda")
    for g in range(a.shape[0]):
        rows = (ids[:, 0] == g).nonzero()[:, 0]
        if len(rows):
            d, _ = ref.lora(x[rows], a[g], b[g], 1.0, y.dtype)
            finite = [torch.where(t.isfinite(), t, torch.zeros_like(t)) for t in (x[rows], a[g], b[g])]
            _, e = ref.lora(*finite, 1.0, y.dtype)
            want[rows] += d
            tol[rows] = e + 2.0 ** -23 * (torch.nan_to_num(d, 0, 0, 0).abs() + e)
    bound = torch.nan_to_num(ref.rounded(torch.nan_to_num(want, 0, 0, 0), tol, y.dtype), 0, 0, 0)
    ref.assert_within(out, want, bound, "out")
    return out, want


@pytest.mark.parametrize("dtype", [BF16, F16])
@pytest.mark.parametrize("T,G,r,H,N", SIZES)
def test_an_element_of_a(T, G, r, H, N, dtype):
    ids, y, x, a, b = data(T, G, r, H, N, dtype)
    ids[0] = 0
    a[0, r - 1, H // 2] = float("-inf")
    out, want = check(ids, y, x, a, b)
    assert out[0].isinf().all() and (ids[:, 0] == 0).sum() == out.isinf().all(1).sum()


@pytest.mark.parametrize("dtype", [BF16, F16])
@pytest.mark.parametrize("T,G,r,H,N", SIZES)
def test_an_element_of_b(T, G, r, H, N, dtype):
    ids, y, x, a, b = data(T, G, r, H, N, dtype)
    ids[0] = 0
    b[0, N - 3, 2] = float("inf")
    b[0, 5, r - 1] = float("-inf")
    # one row whose sums have exactly one 16-bit number's digits, and so no remainder
    x[0] = 0
    x[0, 1] = 1
    out, want = check(ids, y, x, a, b)
    assert out[0, [5, N - 3]].isinf().all() and out[0].isinf().sum() == 2


@pytest.mark.parametrize("dtype", [BF16, F16])
@pytest.mark.parametrize("T,G,r,H,N", SIZES)
def test_an_element_of_x(T, G, r, H, N, dtype):
    ids, y, x, a, b = data(T, G, r, H, N, dtype)
    x[T // 2, 7] = float("inf")
    x[T - 1, H - 1] = float("inf")
    out, want = check(ids, y, x, a.abs(), b.abs())       # sums of one sign: infinite
    assert out[T - 1].isinf().all()
    out, want = check(ids, y, x, a, b)                   # of both: NaN
    assert out[T - 1].isnan().all() or r < 2


@pytest.mark.parametrize("dtype", [BF16, F16])
@pytest.mark.parametrize("T,G,r,H,N", SIZES)
def test_zero_times_infinity(T, G, r, H, N, dtype):
    ids, y, x, a, b = data(T, G, r, H, N, dtype)
    x[0] = 0
    b[:, 3, 4] = float("inf")
    out, want = check(ids, y, x, a, b)
    assert out[0, 3].isnan() and out[0].isnan().sum() == 1


@pytest.mark.parametrize("T,N", [(16, 96), (20000, 2048)])
def test_sums_near_the_largest_number(T, N):
    """Between bf16's largest number and fp32's: a sum of fp32 that rounds to no bf16."""
    import combine_topk_ids_histogram_gb300 as ep
    H, r, m = 2048, 32, 1.9921875
    x, a = torch.zeros(T, H, dtype=BF16, device="cuda"), torch.zeros(1, r, H, dtype=BF16, device="cuda")
    x[:, 0], x[:, 1] = m * 2.0 ** 63, 2.0 ** 63
    a[0, :, 0], a[0, :, 1] = m * 2.0 ** 63, 1.6875 * 2.0 ** 57
    b = torch.zeros(1, N, r, dtype=BF16, device="cuda")
    b[0, :, 3] = 2.0 ** -100
    y = torch.zeros(T, N, dtype=BF16, device="cuda")
    L = ep.dispatch_layout(torch.zeros(T, 1, dtype=torch.int32, device="cuda"), 1)
    out = ep.lora_add(y, x, a, b, L).double()
    want = (m * m * 2.0 ** 126 + 1.6875 * 2.0 ** 120) * 2.0 ** -100
    assert want * 2.0 ** 100 > torch.finfo(BF16).max and ((out - want).abs() <= 2.0 ** -8 * want).all()
