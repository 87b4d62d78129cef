"""Lengths beyond the table, in the append and the attention that follows it: one rule for both."""
import math

import pytest
import torch

import block_sparse_attention_build_b200 as sa
from cached_cases import Case
from test_rotary_gpu import check as check_turned

pytestmark = pytest.mark.gpu

ALL = sa.Pattern(window=1 << 20)


def i32(a):
    return torch.tensor(a, dtype=torch.int32, device="cuda")


@pytest.mark.parametrize("pattern", [ALL, sa.Pattern(window=20, sinks=3), sa.Pattern(window=5, n_global=70),
                                     sa.Pattern(window=2 ** 31 - 1)], ids=["all", "w20s3", "w5g70", "wmax"])
@pytest.mark.parametrize("prefix", [0, 37])
@pytest.mark.parametrize("m", [1, 3, 60])
def test_append_and_attention_beyond_the_table(m, prefix, pattern):
    """Tables of 64 places; sequences that end in them, cross their end, lie behind them, and a negative one."""
    D, Hq, Hkv, page, room = 64, 4, 2, 16, 64
    lens = [64, 64 + (m + 1) // 2, 64 + m, 64 + m + 11, 40 + m, -3, 2 ** 31 - 1]
    B = len(lens)
    c = Case([m] * B, [room] * B, Hq=Hq, Hkv=Hkv, D=D, page=page, prefix=prefix, seed=401)
    c.table = c.table[:, :room // page].contiguous()
    cache = c.cache()
    batch = sa.CacheBatch(c.dev(c.q_start), i32(lens), c.dev(c.table), max_q=m)
    g = torch.Generator().manual_seed(402)
    x = torch.randn(B * m, Hq + 2 * Hkv, D, generator=g).bfloat16().cuda()
    q, k, v = x[:, :Hq], x[:, Hq:Hq + Hkv], x[:, Hq + Hkv:]
    freq = [100.0 ** (-i / 32) for i in range(32)]
    tokens = [min(max(n, 0), 2 ** 29 - 1) for n in lens]
    place = [n - m + i for n in tokens for i in range(m)]
    turned = sa.cache_append(k, v, cache, batch, rotary=sa.Rotary(freq), pos_offset=prefix, q=q)
    check_turned(turned, q, i32(place)[None, :, None] + prefix, freq, [0] * 32, False)
    # the plain form: keys of the tokens that have a place, rows at their positions
    kt = sa.cache_append(k, v, cache, batch, rotary=sa.Rotary(freq), pos_offset=prefix, q=k)  # the turned keys
    pages = cache.k.clone(), cache.v.clone()
    for b in range(B):
        for i in range(m):
            at = place[b * m + i]
            if 0 <= at < room:
                c.k[b][prefix + at], c.v[b][prefix + at] = kt[b * m + i].cpu(), v[b * m + i].cpu()
        c._put(c.table[b].tolist(), c.k[b][prefix:], c.v[b][prefix:])
    assert torch.equal(pages[0].nan_to_num(9.0), c.dev(c.k_pages).nan_to_num(9.0))
    assert torch.equal(pages[1].nan_to_num(9.0), c.dev(c.v_pages).nan_to_num(9.0))
    args = (turned, cache, batch)
    o, lse = (sa.fwd_shared(*args, c.dev(c.prefix_table), prefix, pattern) if prefix else
              sa.fwd_cached(*args, pattern))
    assert sa.check_device() == sa.SA_OK
    scale = 1 / math.sqrt(D)
    for b in range(B):
        n = prefix + min(tokens[b], room)
        p = torch.tensor([prefix + a for a in place[b * m:b * m + m]], device="cuda")[:, None]
        kv = torch.arange(n, device="cuda")[None]
        see = (kv <= p) & ((p - kv <= pattern.window) | (kv < pattern.sinks) | (kv < pattern.n_global)
                           | (p < pattern.n_global))
        for h in range(Hq):
            qh = turned[b * m:b * m + m, h].double()
            kh, vh = c.dev(c.k[b][:n, h // 2]).double(), c.dev(c.v[b][:n, h // 2]).double()
            s = (qh @ kh.T * scale).masked_fill(~see, -math.inf)
            some = see.any(1)
            w = torch.where(some[:, None], torch.softmax(s, 1), 0.0)
            O, A, L = w @ vh, w @ vh.abs(), torch.logsumexp(s, 1)
            got, l = o[b * m:b * m + m, h].double(), lse[b * m:b * m + m, h].double()
            assert torch.equal(torch.isneginf(l), ~some)
            # as Case.check: the scores' part, twice 2^-21 for the exponentials, 2^-8 for the weights and for O
            e_s = (D + 8) * 2.0 ** -24 * scale * qh.norm(dim=1) * (kh.norm(dim=1).max() if n else 0)
            tol = 2.0 ** -8 * O.abs() + (2.0 ** -8 + 2.0 ** -19 + 2 * e_s[:, None]) * (1 + 2.0 ** -7) * A
            assert bool(((got - O).abs() <= tol).all())
            assert bool(((l - L).abs()[some] <= (e_s + 2.0 ** -19 + 2.0 ** -22 * L.abs())[some]).all())
