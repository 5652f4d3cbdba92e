"""Calls of attention over the 4-bit cache for tests: operands, and the definition's result with a bound for each element.

The bound counts roundings. The weights w_j enter the second product rounded to bf16 (2^-8 of each, at most), the
output is rounded to bf16 (2^-8 of it), and exponentials, scores and sums in 32 bits stay within 2^-11 of sum w |v|:
    |got - want| <= 2^-8 |want| + (2^-8 + 2^-11) sum_j w_j |v_j|
"""
import numpy as np
import torch

import kv4_util as K

# With this many promised new tokens the prompts' cache is expanded before, once.
MANY = 1100


def pack(pool, slots, which, c, s, z):
    """Pool.store of many tokens at once: codes [n, Hk, d], pairs [n, Hk, d/32] of different slots."""
    slots = np.asarray(slots, np.int64)
    n, Hk, d, P = len(slots), pool.Hk, pool.d, pool.P
    rec = pool.raw.reshape(pool.n, Hk, -1)
    a, b = P * d // 2, P * d // 8
    pair = torch.from_numpy(np.stack((s, z), -1).reshape(n, Hk, -1).astype(np.float32)).to(torch.bfloat16)
    pair = pair.view(torch.int16).numpy().view(np.uint8).reshape(n, Hk, d // 8)
    page, off = (slots // P)[:, None, None], (slots % P)[:, None, None]
    h = np.arange(Hk)[None, :, None]
    rec[page, h, which * a + off * (d // 2) + np.arange(d // 2)] = c[..., 0::2] | (c[..., 1::2] << 4)
    rec[page, h, 2 * a + which * b + off * (d // 8) + np.arange(d // 8)] = pair


class Case:
    """lens: keys of each sequence, the `new` tokens included. make(b, which, r) gives keys (0) or values (1) of a
    sequence as float32 [len, Hk, d], or None for normal ones; edit_q(q) changes the queries [N, H, d] in place."""

    def __init__(self, lens, new, H, Hk, d, P, seed=0, make=None, edit_q=None, q_scale=1.0, blocks=None, pad=0):
        r = np.random.RandomState(seed)
        self.lens, self.new, self.H, self.Hk, self.d, self.P = lens, new, H, Hk, d, P
        need = [-(-l // P) for l in lens]
        self.n_pages = sum(need) + 2
        self.blocks = blocks or max(need) + 1
        ids, at = r.permutation(self.n_pages), 0
        self.table = np.full((len(lens), self.blocks), -1, np.int32)
        pool = K.Pool(self.n_pages, Hk, d, P, fill=0xFF)  # NaN pairs wherever nothing is stored
        self.kv = []
        for b, l in enumerate(lens):
            self.table[b, :need[b]] = ids[at:at + need[b]]
            at += need[b]
            j = np.arange(l)
            held = []
            for which in (0, 1):
                x = make(b, which, r) if make else None
                c, s, z = K.quantise((r.randn(l, Hk, d) if x is None else x).astype(np.float32))
                pack(pool, self.table[b, j // P] * P + j % P, which, c, s, z)
                held.append(K.values(c, s, z))
            self.kv.append(held)
        self.pool = pool.raw
        self.q_start = np.concatenate(([0], np.cumsum(new)))
        self.N, self.pad = int(self.q_start[-1]), pad
        q = r.randn(self.N + pad, H, d).astype(np.float32) * np.float32(q_scale)
        if edit_q:
            edit_q(q)
        self.q = torch.from_numpy(q).to(torch.bfloat16)

    def operands(self, L, max_new=None, room=None):
        """The arguments of llm_op_attention_kv4; room: bytes of workspace."""
        mx = max(self.new) if max_new is None else max_new
        ask = L.llm_op_attention_kv4_workspace(len(self.lens), self.N + self.pad, mx, self.H, self.Hk, self.d, self.blocks, self.P)
        ws = torch.full((ask if room is None else room,), 255, dtype=torch.uint8, device="cuda")
        dev = lambda a: torch.from_numpy(np.ascontiguousarray(a, np.int32)).cuda()
        out = torch.full((self.N + self.pad, self.H * self.d), -7.0, dtype=torch.bfloat16, device="cuda")
        return [self.q.cuda(), torch.from_numpy(self.pool).cuda(), self.P, self.Hk, dev(self.table), dev(self.lens),
                dev(self.q_start), mx, out, ws]

    def run(self, L, max_new=None, room=None):
        args = self.operands(L, max_new, room)
        torch.cuda.synchronize()
        for _ in range(2):  # the second call finds the first one's leavings in the workspace
            L.llm_op_attention_kv4(*args)
        L.llm_op_synchronize()
        out = args[8].float().cpu().numpy()
        assert (out[self.N:] == -7.0).all()
        return out[:self.N].reshape(self.N, self.H, self.d)

    def want(self, b, drop=None):
        """(result, bound) of a sequence's rows [n, H, d], from the definition in 64 bits; drop: keys left out."""
        k, v = self.kv[b]
        l, n, G = self.lens[b], self.new[b], self.H // self.Hk
        q = self.q[self.q_start[b]:self.q_start[b + 1]].double().numpy()
        seen = np.arange(l)[None] <= (l - n + np.arange(n))[:, None]
        if drop is not None:
            seen[:, drop] = False
        out, bound = np.zeros((n, self.H, self.d)), np.zeros((n, self.H, self.d))
        odd, v = ~np.isfinite(v), np.nan_to_num(v, nan=0.0, posinf=0.0, neginf=0.0)
        for h in range(self.H):
            with np.errstate(all="ignore"):
                s = np.where(seen, q[:, h] @ k[:, h // G].T / np.sqrt(self.d), -np.inf)
                m = s.max(1, keepdims=True)
                w = np.where(seen, np.exp(s - np.where(m == -np.inf, 0, m)), 0.0)
                w /= np.where(m == -np.inf, 1, w.sum(1, keepdims=True))
                out[:, h] = w @ v[:, h // G]
                out[:, h][seen.astype(np.float64) @ odd[:, h // G] > 0] = np.nan  # of the rows that see it
                bound[:, h] = 2.0**-8 * np.abs(np.nan_to_num(out[:, h])) + (2.0**-8 + 2.0**-11) * (w @ np.abs(v[:, h // G]))
        return out, bound

    def check(self, got, rows=None):
        """rows(b): which of a sequence's rows are looked at (all of them)."""
        for b in range(len(self.lens)):
            want, bound = self.want(b)
            g = got[self.q_start[b]:self.q_start[b + 1]]
            if rows is not None:
                at = rows(b)
                g, want, bound = g[at], want[at], bound[at]
            assert np.array_equal(np.isnan(g), np.isnan(want)), b
            over = np.nan_to_num(np.abs(g - want) - bound, nan=0.0)
            assert (over <= 0).all(), (b, over.max(), np.unravel_index(over.argmax(), over.shape))


def marked(Hk, d, lens):
    """make= of a case whose values say which keys were summed: 1 in dimension (j / 16) % d, 0 elsewhere. No terms
    cancel, so the bound of an element is relative to it, and a key more or less shows in it."""
    def make(b, which, r):
        if which == 0:
            return None
        x = np.zeros((lens[b], Hk, d), np.float32)
        j = np.arange(lens[b])
        x[j, :, (j // 16) % d] = 1.0
        return x
    return make
