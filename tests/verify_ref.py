"""Plain form of the verification of drafted tokens: one sequence, one node, one child at a time, in 64 bits."""
import torch


def clean(row):
    row = row.double()
    return torch.where(row > 0, row, torch.zeros_like(row))  # (negative ones and NaN are 0)


def draw(w, u):
    """The smallest token whose running sum is above u times the sum; -1 where all are 0."""
    c = w.cumsum(0)
    if not float(c[-1]) > 0:
        return -1
    above = (c > u * c[-1]).nonzero()[:, 0]
    some = (w > 0).nonzero()[:, 0]
    return int(above[0]) if len(above) else int(some[-1])


def verify(target, tokens, uniform, draft=None, parent=None):
    """(path, count, tokens) of each sequence, and whether any input was refused."""
    paths, counts, outs, flags = [], [], [], False
    for b in range(tokens.shape[0]):
        t, v = tokens.shape[1], target.shape[2]
        up = [i - 1 for i in range(t)] if parent is None else (parent[b] if parent.dim() == 2 else parent).tolist()
        node, path, p = 0, [], clean(target[b, 0])
        w, total, u = p, 1.0, uniform[b].double().tolist()
        for i in range(t):
            x = int(tokens[b, i])
            if not (0 <= x < v and -1 <= up[i] < i):
                flags = True
                continue
            if up[i] != node - 1:
                continue
            q = clean(draft[b, node]) if draft is not None else None
            if u[i] * (total * (float(q[x]) if q is not None else 1.0)) < float(w[x]):
                path.append(i)
                node = i + 1
                p = clean(target[b, node])
                w, total = p, 1.0
            elif q is not None:
                w = (w - total * q).clamp(min=0)
                total = float(w.sum())
            else:
                total -= float(w[x])
                w = w.clone()
                w[x] = 0
        token = draw(w if float(w.sum()) > 0 else p, u[t])
        flags |= token < 0
        paths.append(path + [-1] * (t - len(path)))
        counts.append(len(path))
        outs.append([int(tokens[b, i]) for i in path] + [token] + [-1] * (t - len(path)))
    b, t = tokens.shape
    return (torch.tensor(paths, dtype=torch.int32).reshape(b, t), torch.tensor(counts, dtype=torch.int32),
            torch.tensor(outs, dtype=torch.int64).reshape(b, t + 1), flags)
