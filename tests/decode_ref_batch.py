"""The 64-bit form of the attention for whole batches: decode_ref.attend's outputs by products of matrices, one sequence
and key head at a time, for sizes at which one query row at a time takes too long."""
import math

import torch


def attend(q, key, value, d_v, page_size, table, lens, seqs, cu, scale, mask):
    T, H, _ = q.shape
    Hk = key.shape[2]
    G = H // Hk
    out, lse = torch.zeros(T, H, d_v, dtype=torch.float64), torch.full((T, H), -math.inf, dtype=torch.float64)
    A, D, L = torch.zeros(T, H, d_v, dtype=torch.float64), torch.zeros(T, H, dtype=torch.float64), torch.zeros(T)
    for j, seq in enumerate(seqs):
        n, past = cu[j + 1] - cu[j], lens[seq]
        if n == 0 or past + n == 0:
            continue
        rows = torch.arange(past + n)
        pages = table[seq].long()[rows // page_size]
        see = torch.ones(n, past + n, dtype=torch.bool)
        k = torch.arange(n)
        for i in range(n):
            see[i, past:] = k <= i if mask is None else (mask[cu[j] + i, k // 32] >> (k % 32)) & 1 == 1
        L[cu[j]: cu[j + 1]] = see.sum(1).float()
        for g in range(Hk):
            kk = key[pages, rows % page_size, g]
            vv = value[pages, rows % page_size, g] if value is not None else kk[:, :d_v]
            qq = q[cu[j]: cu[j + 1], g * G: (g + 1) * G].double().reshape(n * G, -1)
            s = (qq @ kk.T * scale).masked_fill(~see.repeat_interleave(G, 0), -math.inf)
            m = s.max(1, keepdim=True).values
            some = torch.isfinite(m[:, 0])
            w = torch.exp(s - m.nan_to_num(0, 0, 0))
            tot = w.sum(1, keepdim=True)
            d = (qq.abs() @ kk.abs().T * abs(scale)).masked_fill(~see.repeat_interleave(G, 0), 0).max(1).values
            put = lambda to, x, off: to[cu[j]: cu[j + 1], g * G: (g + 1) * G].copy_(  # noqa: E731
                torch.where(some.view(-1, *[1] * (x.dim() - 1)), x, off).view(n, G, *x.shape[1:]))
            put(out, w @ vv / tot, 0.0)
            put(A, w @ vv.abs() / tot, 0.0)
            put(lse, (m + torch.log(tot))[:, 0], -math.inf)
            put(D, d, 0.0)
    return out, lse, A, D, L
