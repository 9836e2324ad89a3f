"""nn.linear_distillation refuses tensors whose leading dimensions or entries do not
belong together, which its flat views would lay out anew."""
import pytest


def test_distillation_shapes():
    torch = pytest.importorskip("torch")
    import __graft_entry__
    __graft_entry__.build()
    from bit_optimizer_gb300 import nn

    x, w = torch.zeros(4, 6, 8).half(), torch.zeros(30, 8).half()
    ids = torch.zeros(4, 6, 5).long()

    def refused(x, ids, logits):
        with pytest.raises(ValueError, match="shape"):
            nn.linear_distillation(x, w, ids, logits)
    refused(x, ids, torch.zeros(6, 4, 5))
    refused(x, ids, torch.zeros(4, 5, 6))
    refused(x, ids, torch.zeros(24, 5))
    refused(x, ids, torch.zeros(4, 6, 4))
    refused(x, ids.transpose(0, 1), torch.zeros(6, 4, 5))
    refused(x, ids.view(24, 5), torch.zeros(24, 5))
    refused(x, ids[..., :0], torch.zeros(4, 6, 0))
    refused(x[0, 0], ids[0, 0, 0], torch.zeros(()))
    # what belongs together reaches the operator, which takes CUDA tensors
    for lead in ((4, 6), (24,), (1, 4, 6), ()):
        n = 8 if lead else 1
        with pytest.raises(TypeError, match="CUDA"):
            nn.linear_distillation(torch.zeros(*lead, 8).half(), w, torch.zeros(*lead, n).long(),
                                   torch.zeros(*lead, n))
