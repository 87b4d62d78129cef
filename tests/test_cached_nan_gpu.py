"""NaN and infinite scores in cached attention: a row that sees one has NaN for its output and its LSE, on
every path (items whole in a CTA or cluster, cut over CTAs or warps, over a prefix); the other rows keep
their values."""
import copy
import math

import pytest
import torch

import block_sparse_attention_build_b200 as sa
from cached_cases import NAN, Case

pytestmark = pytest.mark.gpu

ALL = sa.Pattern(window=1 << 20)
WS = sa.Pattern(window=100, sinks=4)

PATHS = {
    "items": lambda: Case([1] * 3, [200, 90, 30], seed=301),
    "clusters": lambda: Case([1], [700], Hq=2, Hkv=2, D=64, seed=302),
    "line": lambda: Case([1] * 3, [20000, 90, 30], seed=303),
    "line of 24 rows": lambda: Case([3] * 2, [9000, 700], Hq=16, Hkv=2, seed=304),
    "warps": lambda: Case([1] * 160, [70 + (53 * b) % 200 for b in range(160)], Hq=8, Hkv=4, seed=305),
    "piece": lambda: Case([1, 300], [200, 900], D=64, seed=306),
    "one piece": lambda: Case([70], [6000], Hq=8, Hkv=2, page=64, seed=307),
    "tails": lambda: Case([700, 1, 900], [5000, 300, 900], Hq=12, Hkv=2, page=64, seed=308),
    "prefix": lambda: Case([1] * 3, [60, 39, 33], prefix=300, seed=309),
    "prefix in parts": lambda: Case([1] * 40, [50] * 40, prefix=300, Hq=8, Hkv=2, seed=310),
    "prefix and join": lambda: Case([1] * 70, [40] * 70, prefix=12000, Hq=8, Hkv=2, page=64, seed=311),
    "prefix and pieces": lambda: Case([150, 1], [300, 40], prefix=500, Hq=4, Hkv=2, page=32, seed=312),
}


def keys_of(c, b, lo, hi, value, k_value):
    """Set keys lo .. hi - 1 (prefix included) of sequence b: `value` in the cache, `k_value` in the plain copy."""
    c.k[b] = c.k[b].clone()
    if lo < c.prefix:  # the prefix's keys are every sequence's
        for i in range(c.B):
            c.k[i] = c.k[i].clone()
            c.k[i][lo:hi] = k_value
        pre = c.k[b][:c.prefix].clone()
        pre[lo:hi] = value
        c._put(c.prefix_table.tolist(), pre, c.v[b][:c.prefix])
    else:
        c.k[b][lo:hi] = k_value
        own = c.k[b][c.prefix:].clone()
        own[lo - c.prefix:hi - c.prefix] = value
        need = -(-c.kv_len[b] // c.page)
        c._put(c.table[b, :need].tolist(), own, c.v[b][c.prefix:])


def poison(c, what):
    """(what the call gets, the same with zeros in place of what is poisoned)"""
    clean = copy.deepcopy(c)
    n = c.prefix + c.kv_len[0]
    if what.startswith("query"):
        value = math.inf if what == "query inf" else NAN
        rows = sorted({0, c.q_len[0] // 2, c.T - 1})
        for t in rows:
            c.q[t, t % c.Hq, 5] = value
            clean.q[t, t % c.Hq, 5] = 0
        return c, clean
    if what == "page":
        lo, hi = n - 40, n - 20
    elif what == "prefix page":
        lo, hi = c.prefix // 2, c.prefix // 2 + 20
    else:  # one key, at a place of its tile whose weight is taken by either kind of exponential
        lo = (n - 30) // 128 * 128 + (16 if what == "key 16" else 17)
        lo = lo if lo < n else lo - 128
        hi = lo + 1
    if lo < c.prefix < hi:
        hi = c.prefix
    for x, plain in ((c, NAN), (clean, 0.0)):
        keys_of(x, 0, lo, hi, NAN, plain)
    return c, clean


def check(c, clean, pattern):
    o, lse = c.run(pattern)
    L = c.plain(pattern)[1]
    O0, L0, _, _ = clean.plain(pattern)
    T = L.shape[0]
    bad = torch.isnan(L) | torch.isposinf(L)
    o, lse = o[:T], lse[:T]
    assert torch.equal(torch.isnan(lse), bad)
    assert torch.equal(torch.isnan(o).all(-1), bad) and torch.equal(torch.isnan(o).any(-1), bad)
    o[bad], lse[bad] = O0[bad].bfloat16(), L0[bad].float()
    clean.check(o, lse, pattern)
    return bad


@pytest.mark.parametrize("pattern", [ALL, WS], ids=["all", "w100s4"])
@pytest.mark.parametrize("what", ["query", "query inf", "page", "key 16", "key 17", "prefix page"])
@pytest.mark.parametrize("path", PATHS)
def test_nan_reaches_the_rows_that_see_it(path, what, pattern):
    c = PATHS[path]()
    if what == "prefix page" and not c.prefix:
        what = "page"
        c.q *= 4  # another distribution of the other rows
    c, clean = poison(c, what)
    bad = check(c, clean, pattern)
    if pattern is ALL or what in ("query", "query inf", "page"):  # the others may lie below the window
        assert bool(bad.any())


def test_a_nan_row_answers_the_same_whole_and_cut():
    """The same sequence alone, where its items are whole, and in batches that cut them."""
    got = []
    for others in (0, 1, 40, 200):
        c = Case([1] * (1 + others), [400] + [1 + 97 * b % 900 for b in range(others)], Hq=8, Hkv=2, seed=321)
        c.q[0, 3, 0] = NAN
        o, lse = c.run(ALL)
        got.append((torch.isnan(o[0]), torch.isnan(lse[0])))
    for a, b in got:
        assert a[3].all() and b[3] and int(a.sum()) == c.D and int(b.sum()) == 1
