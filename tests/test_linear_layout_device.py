"""A layout of another device than the current one is refused, like a tensor there."""
import pytest
import torch


def _ep():
    import __graft_entry__ as entry
    entry._load_builder().build()
    import combine_topk_ids_histogram_gb300 as ep
    return ep


def calls(ep, L, device):
    new = lambda *shape: torch.zeros(*shape, dtype=torch.bfloat16, device=device)
    x, w, g, a, b = new(80, 64), new(2, 96, 64), new(80, 96), new(2, 8, 64), new(2, 64, 8)
    return (lambda: ep.expert_linear(x, w, L), lambda: ep.expert_linear(x, w, L, swiglu=True, save=True), lambda: ep.expert_linear_bwd(g, x, w, L),
            lambda: ep.lora_add(x, x, a, b, L, by_token=False), lambda: ep.lora_add(x, x, a, b, L))


def test_without_a_gpu(monkeypatch):
    """The host's memory as the current device, and a layout that says it is on the first GPU."""
    ep = _ep()
    L = ep.Layout(80, 1, 2, device="cpu")
    L.device_index = 0
    monkeypatch.setattr(torch.cuda, "current_device", lambda: -1)
    for f in calls(ep, L, "cpu"):
        with pytest.raises(ValueError, match="layout"):
            f()


@pytest.mark.gpu
def test_layout_in_host_memory():
    import combine_topk_ids_histogram_gb300 as ep
    L = ep.Layout(80, 1, 2, device="cpu")
    for f in calls(ep, L, "cuda"):
        with pytest.raises(ValueError, match="layout"):
            f()
