"""Inputs of the cached-attention tests and their plain implementation in 64 bits."""
import math

import torch

import block_sparse_attention_build_b200 as sa

NAN = float("nan")


class Case:
    """A batch over a paged cache.  Places that hold no token, and pages of no sequence, are NaN or
    infinite; table entries behind a sequence's pages are out of range."""

    def __init__(self, q_len, kv_len, Hq=4, Hkv=2, D=128, page=16, prefix=0, token_major=False, seed=0, pad_rows=0,
                 device="cuda", q_scale=1.0):
        g = torch.Generator().manual_seed(seed)
        rnd = lambda *s: torch.randn(*s, generator=g).to(torch.bfloat16)
        self.q_len, self.kv_len, self.Hq, self.Hkv, self.D, self.page = q_len, kv_len, Hq, Hkv, D, page
        self.prefix, self.B, self.device = prefix, len(q_len), device
        self.T = sum(q_len) + pad_rows
        need = [-(-max(n, 0) // page) for n in kv_len]
        n_pre = -(-prefix // page)
        n_pages = sum(need) + n_pre + 2
        order = torch.randperm(n_pages, generator=g).tolist()
        shape = (n_pages, page, Hkv, D) if token_major else (n_pages, Hkv, page, D)
        k, v = torch.full(shape, NAN, dtype=torch.bfloat16), torch.full(shape, math.inf, dtype=torch.bfloat16)
        self.k_pages, self.v_pages = (x.transpose(1, 2) if token_major else x for x in (k, v))
        self.table = torch.full((self.B, max(need + [1]) + 1), -7, dtype=torch.int32)
        self.table[:, -1] = n_pages + 5
        self.prefix_table = torch.tensor(order[:n_pre], dtype=torch.int32)
        at = n_pre
        self.k, self.v = [], []  # per sequence: [prefix + kv_len, Hkv, D]
        kp, vp = rnd(prefix, Hkv, D), rnd(prefix, Hkv, D)
        self._put(order[:n_pre], kp, vp)
        for b, n in enumerate(kv_len):
            n = max(n, 0)
            pages = order[at:at + need[b]]
            at += need[b]
            self.table[b, :need[b]] = torch.tensor(pages, dtype=torch.int32)
            kb, vb = rnd(n, Hkv, D), rnd(n, Hkv, D)
            self._put(pages, kb, vb)
            self.k.append(torch.cat([kp, kb]))
            self.v.append(torch.cat([vp, vb]))
        self.q = rnd(self.T, Hq, D) * q_scale
        self.q_start = torch.tensor([sum(q_len[:b]) for b in range(self.B + 1)], dtype=torch.int32)

    def _put(self, pages, k, v):
        for i, pg in enumerate(pages):
            a, z = i * self.page, min((i + 1) * self.page, k.shape[0])
            self.k_pages[pg, :, :z - a] = k[a:z].transpose(0, 1)
            self.v_pages[pg, :, :z - a] = v[a:z].transpose(0, 1)

    def dev(self, x):
        return x.to(self.device)

    def cache(self):
        # .to keeps a dense tensor's strides
        return sa.KVCache(self.dev(self.k_pages), self.dev(self.v_pages))

    def batch(self, max_q=None):
        return sa.CacheBatch(self.dev(self.q_start), self.dev(torch.tensor(self.kv_len, dtype=torch.int32)),
                             self.dev(self.table), max_q=max_q)

    def run(self, pattern, max_q=None, scale=None, **kw):
        args = (self.dev(self.q), self.cache(), self.batch(max_q if max_q is not None else max(self.q_len + [0])))
        if self.prefix:
            o, l = sa.fwd_shared(*args, self.dev(self.prefix_table), self.prefix, pattern, scale=scale, **kw)
        else:
            o, l = sa.fwd_cached(*args, pattern, scale=scale, **kw)
        assert sa.check_device() == sa.SA_OK
        return o, l

    def plain(self, pattern, scale=None):
        """(O, LSE, sum of p |v|, bound on |q| . |k|) in 64 bits for the rows of the sequences."""
        scale = scale if scale is not None else 1 / math.sqrt(self.D)
        dev = self.device
        T = int(self.q_start[-1])
        O = torch.zeros(T, self.Hq, self.D, dtype=torch.float64, device=dev)
        A = torch.zeros_like(O)
        L = torch.full((T, self.Hq), -math.inf, dtype=torch.float64, device=dev)
        S = torch.zeros((T, self.Hq), dtype=torch.float64, device=dev)
        G = self.Hq // self.Hkv
        for b in range(self.B):
            m, n = self.q_len[b], self.prefix + max(self.kv_len[b], 0)
            if m == 0 or n == 0:
                continue
            t0 = int(self.q_start[b])
            p = torch.arange(n - m, n, device=dev)[:, None]
            kv = torch.arange(n, device=dev)[None]
            see = (kv <= p) & (((p - kv <= pattern.window) if pattern.window >= 0 else (kv < 0)) | (kv < pattern.sinks)
                               | (kv < pattern.n_global) | (p < pattern.n_global))
            k, v = self.dev(self.k[b]).double(), self.dev(self.v[b]).double()
            q = self.dev(self.q[t0:t0 + m]).double()
            for h in range(self.Hq):
                kh, vh, qh = k[:, h // G], v[:, h // G], q[:, h]
                x = (qh @ kh.T * scale).masked_fill(~see, -math.inf)
                some = see.any(1)
                w = torch.where(some[:, None], torch.softmax(x, 1), 0.0)
                O[t0:t0 + m, h] = w @ vh
                A[t0:t0 + m, h] = w @ vh.abs()
                L[t0:t0 + m, h] = torch.logsumexp(x, 1)
                S[t0:t0 + m, h] = scale * qh.norm(dim=1) * kh.norm(dim=1).max()
        return O, L, A, S

    def check(self, o, lse, pattern, scale=None):
        """Against the plain implementation.  Bounds, all first order:
        scores: D products and sums in 32 bits, each off by 2^-24 of |q| |k| at most -> e_s; one weight
        is then off by a factor 1 + 2 e_s (its own and the denominator's), by 2^-21 twice for the
        exponential (2^x on either pipe is within 2.3e-7) and by 2^-8 for its rounding to bf16 before
        P V; O is rounded to bf16 (2^-8 of itself), and partial results are joined in 32 bits, each join
        with two more exponentials.  The LSE adds the logarithm (2^-21) and its own rounding."""
        O, L, A, S = self.plain(pattern, scale)
        T = O.shape[0]
        o, lse = o[:T].double(), lse[:T].double()
        e_s = (self.D + 8) * 2.0 ** -24 * S
        none = torch.isneginf(L)
        assert torch.equal(torch.isneginf(lse), none)
        assert bool((o[none] == 0).all()) and bool(torch.isfinite(o).all())
        tol = 2.0 ** -8 * O.abs() + (2.0 ** -8 + 2.0 ** -19 + 2 * e_s[..., None]) * (1 + 2.0 ** -7) * A
        over = (o - O).abs() - tol
        assert bool((over <= 0).all()), f"O off by {float((o - O).abs().max())}, {float(over.max())} over its bound"
        l_off = (lse - L).abs()[~none]
        l_tol = (e_s + 2.0 ** -19 + 2.0 ** -22 * L.abs())[~none]
        assert bool((l_off <= l_tol).all()), f"LSE off by {float(l_off.max())}"
