"""The adapters read the layout before they know its status: whatever a layout with a status holds, nothing is written, nothing outside
the buffers is touched, and the status stays what it was."""
import pytest
import torch

import linear_ref as ref

pytestmark = pytest.mark.gpu

BF16 = torch.bfloat16
BIG = 2 ** 31 - 1


def fill(L, value):
    for t in (L.row_offsets, L.expert_ids, L.src_info, L.row_of):
        if value is None:
            g = torch.Generator().manual_seed(1)
            t.copy_(torch.randint(-BIG, BIG, t.shape, generator=g, dtype=torch.int32))
        else:
            t.fill_(value)


@pytest.mark.parametrize("T,G,r,H,N", [(1, 3, 16, 64, 48), (40, 3, 24, 2048, 96), (9000, 2, 72, 2560, 496)])
@pytest.mark.parametrize("value", [None, -1, 0, 1, BIG, -BIG])
@pytest.mark.parametrize("status", ["BAD_EXPERT", "OVERFLOW", "TIMEOUT"])
def test_anything_in_a_layout_with_a_status(T, G, r, H, N, value, status):
    import combine_topk_ids_histogram_gb300 as ep
    bit = getattr(ep, "STATUS_" + status)
    normal = lambda *shape: torch.randn(*shape, device="cuda").to(BF16)
    x, y, a, b = normal(T, H), normal(T, N), normal(G, r, H), normal(G, N, r)
    for by_token in (True, False):
        L = ep.dispatch_layout(torch.zeros(T, 1, dtype=torch.int32, device="cuda"), G)
        fill(L, value)
        L.status.fill_(bit)
        buf = torch.full((T * N + 4096,), 7.0, dtype=BF16, device="cuda")
        ep.lora_add(y, x, a, b, L, by_token=by_token, out=buf[:T * N].view(T, N))
        torch.cuda.synchronize()
        assert (buf == 7).all()
        assert L.status[0].item() == bit


@pytest.mark.parametrize("swiglu", [False, True])
def test_products_too(swiglu):
    import combine_topk_ids_histogram_gb300 as ep
    for value in (None, -1, BIG, -BIG):
        L = ref.layout_of(ep, [10, 20, 30])
        fill(L, value)
        L.status.fill_(ep.STATUS_TIMEOUT)
        x, w = torch.randn(60, 64, device="cuda").to(BF16), torch.randn(3, 96, 64, device="cuda").to(BF16)
        buf = torch.full((60 * 96 + 4096,), 7.0, dtype=BF16, device="cuda")
        n = 48 if swiglu else 96
        ep.expert_linear(x, w, L, swiglu=swiglu, out=buf[:60 * n].view(60, n))
        gw = torch.full((3, 96, 64), 7.0, dtype=BF16, device="cuda")
        gx = torch.full((60, 64), 7.0, dtype=BF16, device="cuda")
        ep.expert_linear_bwd(torch.randn(60, 96, device="cuda").to(BF16), x, w, L, out=(gx, gw))
        torch.cuda.synchronize()
        assert all((t == 7).all() for t in (buf, gx, gw))
        assert L.status[0].item() in (ep.STATUS_TIMEOUT, ep.STATUS_TIMEOUT | ep.STATUS_BOUNDS)
