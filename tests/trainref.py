"""64-bit references of the vocabulary loss, the sorted rows and the clipping, and inputs whose logits are exact."""
import torch


def gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def exact_head(T, H, V, seed, spread=4.0):
    """x [T,H] and W [V,H] bf16 whose products add up without rounding in any order: x in {-1, 0, 1}, W multiples of
    1/32, so every partial sum is a multiple of 1/32 below 2^16. Logits of about `spread`."""
    g = gen(seed)
    x = torch.randint(-1, 2, (T, H), generator=g, device="cuda").to(torch.bfloat16)
    std = max(32 * spread / (H * 2 / 3) ** 0.5, 0.7)
    W = (torch.randn((V, H), generator=g, device="cuda") * std).round().clamp(-128, 128) / 32
    return x, W.to(torch.bfloat16)


def head_loss(x, W, labels):
    """(loss, lse, live) in 64 bits; the loss from the other tokens' share."""
    V = W.shape[0]
    l = x.double() @ W.double().t()
    live = (labels >= 0) & (labels < V)
    col = torch.where(live, labels.long(), 0)[:, None]
    lse = torch.logsumexp(l, 1)
    at = l.gather(1, col)[:, 0]
    rest = torch.logsumexp(l.scatter(1, col, float("-inf")), 1)
    loss = torch.nn.functional.softplus(rest - at, threshold=200.0)
    zero = torch.zeros_like(loss)
    return torch.where(live, loss, zero), torch.where(live, lse, zero), live


def head_grad(x, W, labels, coef):
    """(dx, dW, sum |dl||W|, sum |dl||x|) in 64 bits for the loss sum(coef * loss)."""
    xd, Wd = x.double(), W.double()
    l = xd @ Wd.t()
    live = (labels >= 0) & (labels < W.shape[0])
    col = torch.where(live, labels.long(), 0)[:, None]
    p = torch.softmax(l, 1)
    rest = torch.logsumexp(l.scatter(1, col, float("-inf")), 1)
    p = p.scatter(1, col, -torch.exp(rest - torch.logsumexp(l, 1))[:, None])
    dl = torch.where(live[:, None], coef[:, None] * p, 0.0)
    xd = torch.where(live[:, None], xd, 0.0)
    return dl @ Wd, dl.t() @ xd, dl.abs() @ Wd.abs(), dl.abs().t() @ xd.abs()


def layout(idx, E):
    """counts, offsets, row_src, slot_row of a list of lists of expert indices."""
    flat = [e for row in idx for e in row]
    kept = sorted((i for i, e in enumerate(flat) if 0 <= e < E), key=lambda i: (flat[i], i))
    counts = [sum(1 for i in kept if flat[i] == e) for e in range(E)]
    offsets = [sum(counts[:e]) for e in range(E + 1)]
    slot = [-1] * len(flat)
    for r, i in enumerate(kept):
        slot[i] = r
    return counts, offsets, kept + [-1] * (len(flat) - len(kept)), slot
