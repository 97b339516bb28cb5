"""Which outs hold a tensor's values in the same order (CPU)."""
import torch

import cross_entropy_loss_ce_gb300 as gbce


def test_same_order_of_values():
    x = torch.zeros(4, 6, 5)
    for t, o in ((x, x), (x, torch.zeros(120)), (x.permute(2, 0, 1), torch.zeros(4, 6, 5).permute(2, 0, 1)),
                 (torch.zeros(1, 8, 5).transpose(1, 2), torch.zeros(8, 5).t()[None]),
                 (x[:1].transpose(0, 2), torch.zeros(6, 5).t()[:, :, None]), (x[:, :0], torch.zeros(0)),
                 (torch.zeros(()), torch.zeros(1))):
        assert gbce._same_order(t, o) and gbce._same_order(o, t)
    for t, o in ((x.permute(2, 0, 1), x.permute(2, 1, 0)), (x.permute(2, 0, 1), torch.zeros(5, 4, 6)),
                 (torch.zeros(6, 4).t(), torch.zeros(4, 6)), (torch.zeros(6, 4).t(), torch.zeros(24)),
                 (torch.zeros(4, 4).t(), torch.zeros(4, 4))):
        assert not gbce._same_order(t, o) and not gbce._same_order(o, t)
