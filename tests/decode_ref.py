"""Plain 64-bit forms of the decode-side operators, on the CPU: what the GPU
tests compare against. Written from the formulas in include/mla_qup.h, one
sequence, token and page at a time; nothing is shared with the library."""
import math

import numpy as np
import torch

E2M1 = np.array([0, 0.5, 1, 1.5, 2, 3, 4, 6, -0.0, -0.5, -1, -1.5, -2, -3, -4, -6])


def e4m3_values(codes):
    return codes.view(torch.float8_e4m3fn).double()


def scale_values(scales):
    """2^(byte - 127), NaN for 0xFF."""
    s = torch.exp2(scales.double() - 127)
    return torch.where(scales == 255, torch.nan, s)


def mx8_values(codes, scales):
    return e4m3_values(codes) * scale_values(scales).repeat_interleave(32, -1)


def mx4_values(codes, scales):
    """codes uint8 [N, K/2], scales uint8 [N, K/32] -> [N, K]."""
    c = torch.stack([codes & 15, codes >> 4], -1).flatten(-2).long()
    return torch.from_numpy(E2M1)[c] * scale_values(scales).repeat_interleave(32, -1)


def mx4_quantize(x):
    """(codes [N, K/2], scales [N, K/32]) by search over the 16 values, ties to the even code; x float64 holding
    float32 values."""
    x = x.numpy()
    N, K = x.shape
    codes, scales = np.zeros((N, K), np.uint8), np.zeros((N, K // 32), np.uint8)
    for r in range(N):
        for b in range(K // 32):
            v = x[r, 32 * b: 32 * b + 32]
            if not np.isfinite(v).all():
                codes[r, 32 * b: 32 * b + 32], scales[r, b] = 7, 255
                continue
            amax = np.abs(v).max()
            e = -127 if amax == 0 else min(127, max(-127, math.floor(math.log2(amax)) - 2))
            scales[r, b] = e + 127
            m = np.minimum(np.abs(v) * 2.0 ** -e, 6)
            d = np.abs(m[:, None] - E2M1[None, :8])
            best = d.min(1)
            for k in range(32):
                near = [c for c in range(8) if d[k, c] == best[k]]
                c = near[0] if len(near) == 1 else next(c for c in near if c % 2 == 0)
                codes[r, 32 * b + k] = c | (8 if np.signbit(v[k]) else 0)
    codes = torch.from_numpy(codes)
    return codes[:, 0::2] | (codes[:, 1::2] << 4), torch.from_numpy(scales)


def cache_values(bufs, mx):
    """Key and (or None) value buffers [pages, page, heads, width] in 64 bits."""
    if mx:
        out = [mx8_values(bufs[k], bufs[k + 1]) for k in range(0, len(bufs), 2)]
    else:
        out = [b.double() for b in bufs]
    return out[0], (out[1] if len(out) > 1 else None)


def attend(q, key, value, d_v, page_size, table, lens, seqs, cu, scale, mask):
    """out, lse, and per element what the error bound needs: A = sum_r w_r |value_r| and D = max over the rows seen
    of scale sum |q k| (a bound on what score roundings scale with). key/value: [pages, page, heads, width]."""
    T, H, d_k = q.shape
    Hk = key.shape[2]
    G = H // Hk
    out, lse = torch.zeros(T, H, d_v, dtype=torch.float64), torch.full((T, H), -math.inf, dtype=torch.float64)
    A, D, L = torch.zeros(T, H, d_v, dtype=torch.float64), torch.zeros(T, H, dtype=torch.float64), torch.zeros(T)
    for j, seq in enumerate(seqs):
        n, past = cu[j + 1] - cu[j], lens[seq]
        rows = [(int(table[seq, r // page_size]), r % page_size) for r in range(past + n)]
        if not rows:
            continue
        pg, rr = torch.tensor([a for a, _ in rows]), torch.tensor([b for _, b in rows])
        k = key[pg, rr]
        v = value[pg, rr] if value is not None else k[..., :d_v]
        for i in range(n):
            t = cu[j] + i
            see = [r for r in range(past + n) if r < past or
                   (r - past <= i if mask is None else (int(mask[t, (r - past) // 32]) >> ((r - past) % 32)) & 1)]
            if not see:
                continue
            ks, vs = k[see], v[see]
            L[t] = len(see)
            for h in range(H):
                kk, vv = ks[:, h // G], vs[:, h // G]
                prod = kk * q[t, h].double()
                s = prod.sum(1) * scale
                m = s.max()
                w = torch.exp(s - m)
                tot = w.sum()
                out[t, h] = (w[:, None] * vv).sum(0) / tot
                lse[t, h] = m + torch.log(tot)
                A[t, h] = (w[:, None] * vv.abs()).sum(0) / tot
                D[t, h] = (prod.abs().sum(1) * abs(scale)).max()
    return out, lse, A, D, L


class Pages:
    """The bookkeeping of mla_pool with lists: one call after the other, one entry after the other."""

    def __init__(self, num_pages, page, max_seqs, max_pages, rows):
        self.page, self.num_pages, self.max_seqs, self.max_pages = page, num_pages, max_seqs, max_pages
        self.refs = [0] * num_pages
        self.table = [[] for _ in range(max_seqs)]
        self.lens = [0] * max_seqs
        self.rows = rows  # list of numpy arrays [num_pages, page, ...], one per buffer

    def _first(self, seqs):
        seen, out = set(), []
        for i, s in enumerate(seqs):
            if 0 <= s < self.max_seqs and s not in seen:
                seen.add(s)
                out.append((i, s))
        return out

    def reserve(self, seqs, new):
        free = [p for p in range(self.num_pages) if self.refs[p] == 0]
        refs, plan, at = list(self.refs), [], 0
        for i, s in self._first(seqs):
            rows = self.lens[s] + new[i]
            if new[i] < 0 or rows > self.max_pages * self.page:
                return -1
        for i, s in self._first(seqs):
            rows, k = self.lens[s] + new[i], self.lens[s] // self.page
            copy = new[i] > 0 and self.lens[s] % self.page != 0 and refs[self.table[s][k]] > 1
            if copy:
                refs[self.table[s][k]] -= 1
            add = max(0, -(-rows // self.page) - len(self.table[s]))
            plan.append((s, k if copy else None, add))
            at += add + copy
        if at > len(free):
            return at - len(free)
        for s, k, add in plan:
            if k is not None:
                old, p = self.table[s][k], free.pop(0)
                self.refs[old] -= 1
                self.refs[p] = 1
                self.table[s][k] = p
                for b in self.rows:
                    b[p, : self.lens[s] % self.page] = b[old, : self.lens[s] % self.page]
            for _ in range(add):
                p = free.pop(0)
                self.refs[p] = 1
                self.table[s].append(p)
        return 0

    def fork(self, src, dst):
        seen = set()
        for s, d in zip(src, dst):
            ok = 0 <= s < self.max_seqs and 0 <= d < self.max_seqs and d not in seen and s not in dst
            seen.add(d)
            if not ok or self.table[d]:
                continue
            self.table[d] = self.table[s][: -(-self.lens[s] // self.page)]
            self.lens[d] = self.lens[s]
            for p in self.table[d]:
                self.refs[p] += 1

    def free(self, seqs, keep=None):
        for i, s in self._first(seqs):
            left = 0 if keep is None else max(0, min(keep[i], self.lens[s]))
            n = -(-left // self.page)
            for p in self.table[s][n:]:
                self.refs[p] -= 1
            self.table[s] = self.table[s][:n]
            self.lens[s] = left

    def compact(self):
        used = sum(r > 0 for r in self.refs)
        src = [p for p in range(used, self.num_pages) if self.refs[p] > 0]
        dst = [p for p in range(used) if self.refs[p] == 0]
        for s, d in zip(src, dst):
            self.refs[d], self.refs[s] = self.refs[s], 0
            for b in self.rows:
                b[d] = b[s]
            for t in self.table:
                t[:] = [d if p == s else p for p in t]
        return used

    def copy(self, dst, src_ids, dst_ids):
        """Whole pages into `dst` (self or another)."""
        before = [b.copy() for b in self.rows]
        seen = set()
        for s, d in zip(src_ids, dst_ids):
            ok = 0 <= s < self.num_pages and 0 <= d < dst.num_pages and d not in seen
            seen.add(d)
            if ok and not (dst is self and d in src_ids):
                for a, b in zip(before, dst.rows):
                    b[d] = a[s]

    def at(self, s, r):
        return self.table[s][r // self.page], r % self.page

    def accept(self, seqs, path, n_acc):
        for i, s in self._first(seqs):
            n = n_acc[i]
            p = list(path[i][:n]) if 0 <= n <= len(path[i]) else [-1]
            room = len(self.table[s]) * self.page - self.lens[s]
            if any(x < 0 or x >= room for x in p) or any(b <= a for a, b in zip(p, p[1:])):
                continue
            for b in self.rows:
                for a, x in enumerate(p):
                    b[self.at(s, self.lens[s] + a)] = b[self.at(s, self.lens[s] + x)]
            self.lens[s] += n
