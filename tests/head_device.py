"""The output head's losses in 64 bits with torch, on the device of the inputs, for sizes at which a loop over
tokens on the host takes too long.  Targets are (ids, q) per token, as in oracle/head.py."""
import torch


def label_targets(labels, vocab):
    on = (labels >= 0) & (labels < vocab)
    return torch.where(on, labels, 0).long()[:, None], on[:, None].double()


def teacher_targets(ids, logits, vocab, lse=None, scale=1.0):
    on = (ids >= 0) & (ids < vocab)
    a = torch.where(on, scale * logits.double(), -torch.inf)
    norm = torch.logsumexp(a, 1) if lse is None else lse.double()
    q = torch.where(on, torch.exp(a - torch.where(on.any(1), norm, 0.0)[:, None]), 0.0)
    return torch.where(on, ids, 0).long(), torch.nan_to_num(q)


def forward(x, w, ids, q, scale=1.0):
    """(loss, lse, z of the entries, z): 0, -inf and 0 for a token without an entry of q > 0."""
    live = (q > 0).any(1)
    z = scale * (torch.where(live[:, None], x, 0).double() @ w.double().t())
    lse = torch.logsumexp(z, 1)
    at = z.gather(1, ids)
    loss = torch.where(q > 0, q * (torch.log(q.clamp(min=1e-300)) - at + lse[:, None]), 0.0).sum(1)
    return torch.where(live, loss, 0.0), torch.where(live, lse, -torch.inf), torch.where(live[:, None], at, 0.0), z


def logit_gradient(z, ids, q, dloss, dlse, scale=1.0):
    """(g [T, V], size): scale ((dloss Q + dlse) p - dloss q), and the sum of its two terms' magnitudes; rows
    without a target zero."""
    live = (q > 0).any(1)
    dloss, dlse = torch.where(live, dloss.double(), 0.0), torch.where(live, dlse.double(), 0.0)
    g = torch.softmax(z, 1).mul_((scale * (dloss * q.sum(1) + dlse))[:, None])
    term = scale * dloss[:, None] * torch.where(live[:, None], q, 0.0)
    size = g.abs().scatter_add_(1, ids, term.abs())
    return g.scatter_add_(1, ids, -term), size
