"""Paths that only larger or unusual calls take: many rows whose cut items are joined from the CTAs' tail
slots, global rows behind a prefix, calls of two host threads at once."""
import threading

import pytest
import torch

import block_sparse_attention_build_b200 as sa
from cached_cases import Case

pytestmark = pytest.mark.gpu

ALL = sa.Pattern(window=1 << 20)
WS = sa.Pattern(window=700, sinks=70)


def go(case, pattern, **kw):
    T = int(case.q_start[-1])
    out = torch.full((case.T, case.Hq, case.D), 3.0, dtype=torch.bfloat16, device="cuda")
    lse = torch.full((case.T, case.Hq), 5.0, device="cuda")
    o, l = case.run(pattern, out=out, lse=lse, **kw)
    case.check(o, l, pattern)
    assert bool((o[T:] == 3).all()) and bool((l[T:] == 5).all())  # rows of no sequence
    return o[:T], l[:T]


# more than 16384 rows (tokens x heads): one sequence; several; single tokens over long caches between pieces
# (both kernels leave tails); few rows over very long caches, cut over many CTAs; one token more than a row block
MANY_ROWS = [([1050], [6000], 16, 4), ([700, 1, 900], [5000, 300, 900], 12, 2),
             ([1, 500, 1, 1, 600, 1], [9000, 700, 12000, 3, 2500, 7000], 16, 2), ([2060], [2060], 8, 8),
             ([1, 40, 1] + [16] * 41, [20000, 30000, 9] + [16] * 41, 24, 8), ([513, 129], [513, 4000], 33, 1)]


@pytest.mark.parametrize("pad", [0, 40])
@pytest.mark.parametrize("pattern", [ALL, WS], ids=["all", "w700s70"])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("case", MANY_ROWS, ids=[f"rows{i}" for i in range(len(MANY_ROWS))])
def test_many_rows(case, D, pattern, pad):
    q_len, kv_len, Hq, Hkv = case
    c = Case(q_len, kv_len, Hq=Hq, Hkv=Hkv, D=D, page=64, pad_rows=pad, seed=501)
    assert c.T * Hq > 16384
    a, b = go(c, pattern), go(c, pattern)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


@pytest.mark.parametrize("D", [64, 128])
def test_either_side_of_many_rows(D):
    """1024 tokens of 16 heads are joined row by row, with one row of no sequence more by the slots."""
    got = []
    for pad in (0, 1):
        c = Case([1, 623, 400], [8000, 5000, 900], Hq=16, Hkv=4, D=D, page=64, seed=502)
        q = torch.cat([c.q, c.q[:pad]])
        c.q, c.T = q, c.T + pad
        got.append(go(c, WS))
    # the same parts in the same order, added by different code: 32-bit sums of up to 2^5 parts apart
    (o1, l1), (o2, l2) = got
    step = 2.0 ** -8 * torch.maximum(o1.abs(), o2.abs()).float() * 2  # the roundings to bf16 on either side
    assert bool(((o1.float() - o2.float()).abs() <= step + 2.0 ** -18).all())
    assert bool(((l1 - l2).abs() <= 2.0 ** -21 * (1 + l1.abs())).all())


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("n_global", [1, 90, 300, 2000])
@pytest.mark.parametrize("lengths,prefix", [(([1] * 3, [20, 9, 3]), 250), (([1] * 40, [30] * 40), 250),
                                            (([1, 0, 6, 1], [5, 3, 6, 0]), 95), (([150, 1, 40], [300, 20, 40]), 280),
                                            (([200, 3], [200, 3]), 17), (([1] * 40, list(range(1, 41))), 1500)],
                         ids=["ones", "many", "ragged", "piece", "short", "long"])
def test_global_rows_behind_a_prefix(lengths, prefix, n_global, D):
    """Positions, columns and global rows count the prefix; n_global ends within it, behind it, at no row."""
    for Hq, Hkv in ((4, 4), (8, 2)):
        c = Case(*lengths, Hq=Hq, Hkv=Hkv, D=D, page=32, prefix=prefix, seed=503)
        go(c, sa.Pattern(window=30, n_global=n_global))
        go(c, sa.Pattern(window=-1, sinks=120, n_global=n_global))


def test_two_host_threads():
    """Calls of two threads, a stream and a workspace each, give what they give alone."""
    cases = [Case([1] * 9 + [140], [3000, 1, 40, 77, 600, 5000, 2, 64, 128, 900], Hq=8, Hkv=2, seed=504),
             Case([1] * 5, [60, 3, 9, 200, 31], Hq=8, Hkv=2, prefix=600, seed=505)]
    args = [(c.dev(c.q), c.cache(), c.batch(max(c.q_len)), c.dev(c.prefix_table)) for c in cases]
    news = [torch.randn(c.T, 2, c.D, device="cuda").bfloat16() for c in cases]
    spec = sa.Rotary([10000.0 ** (-i / 64) for i in range(64)])

    def call(i, stream=None):
        q, cache, batch, pt = args[i]
        c = cases[i]
        q = sa.cache_append(news[i], news[i], cache, batch, rotary=spec, q=q, stream=stream)
        return (sa.fwd_shared(q, cache, batch, pt, c.prefix, ALL, stream=stream) if c.prefix else
                sa.fwd_cached(q, cache, batch, ALL, stream=stream))

    want = [call(i) for i in range(2)]
    torch.cuda.synchronize()
    got, errors = [[], []], []

    def work(i):
        try:
            stream = torch.cuda.Stream()
            with torch.cuda.stream(stream):
                for _ in range(50):
                    got[i].append(call(i, stream))
            stream.synchronize()
        except Exception as e:  # a thread's exception would go unseen
            errors.append(e)

    threads = [threading.Thread(target=work, args=(i,)) for i in range(2)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not errors
    assert sa.check_device() == sa.SA_OK
    for i in range(2):
        assert len(got[i]) == 50
        for a, b in got[i]:
            assert torch.equal(a, want[i][0]) and torch.equal(b, want[i][1])


# (q_len, kv_len, Hq, Hkv, prefix): sequences a CTA each beside clusters over the prefix, several to a CTA; in the
# prefix's clusters; up to 16 rows in all, and up to 32; no token, no key, padded sequences
BOTH = [([1] * 8, [128, 1, 77, 30, 0, 64, 65, 3], 16, 16, 2043), ([1], [600], 2, 2, 1500), ([1, 1], [300, 40], 8, 1, 900),
        ([1] * 8, [9 * b for b in range(8)], 32, 8, 1000), ([4, 3, 0, 1], [200, 3, 9, 60], 8, 4, 300),
        ([16], [16], 2, 1, 64), ([2, 5], [2, 5], 4, 1, 17), ([1] * 31, [1 + b for b in range(31)], 3, 3, 130)]


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("pattern", [ALL, sa.Pattern(window=150, sinks=5), sa.Pattern(window=3, n_global=40)],
                         ids=["all", "w150s5", "w3g40"])
@pytest.mark.parametrize("case", BOTH, ids=[f"both{i}" for i in range(len(BOTH))])
def test_short_prefixes_beside_their_sequences(case, pattern, D):
    """Few rows in all behind a prefix of few keys: both passes in one launch, captured and replayed too."""
    q_len, kv_len, Hq, Hkv, prefix = case
    c = Case(q_len, kv_len, Hq=Hq, Hkv=Hkv, D=D, page=32, prefix=prefix, pad_rows=1, seed=506)
    o, lse = go(c, pattern)
    args = (c.dev(c.q), c.cache(), c.batch(max(q_len)), c.dev(c.prefix_table), prefix, pattern)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        got = [sa.fwd_shared(*args) for _ in range(2)]  # a workspace each, out of the graph's pool
    for _ in range(2):
        g.replay()
        torch.cuda.synchronize()
        for a, b in got:
            assert torch.equal(a[:len(o)], o) and torch.equal(b[:len(lse)], lse)
