"""GPU parity of attention over the paged cache, single tokens to long pieces, with and without a
shared prefix, against a plain implementation in 64 bits."""
import math

import pytest
import torch

import block_sparse_attention_build_b200 as sa
from cached_cases import Case

pytestmark = pytest.mark.gpu

ALL = sa.Pattern(window=1 << 20)
WS = sa.Pattern(window=100, sinks=4)


def go(case, pattern, scale=None, **kw):
    o, lse = case.run(pattern, scale=scale, **kw)
    case.check(o, lse, pattern, scale)
    return o, lse


# (q_len, kv_len): one token, lengths of zero and one, page and tile borders, mixed batches
LENGTHS = [
    ([1], [1]),
    ([1], [700]),
    ([1] * 5, [1, 15, 16, 17, 300]),
    ([1, 0, 1, 1], [64, 9, 0, 129]),
    ([1] * 3, [2000, 3, 513]),
    ([2, 5, 3], [2, 70, 1025]),
    ([17, 1, 40], [17, 400, 333]),
    ([130], [130]),
    ([200, 1, 300, 0], [900, 257, 300, 40]),
]


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("pattern", [ALL, WS, sa.Pattern(window=0, sinks=1), sa.Pattern(window=-1, sinks=3),
                                     sa.Pattern(window=64, n_global=20), sa.Pattern(window=150, sinks=200)],
                         ids=["all", "w100s4", "w0s1", "s3", "w64g20", "w150s200"])
@pytest.mark.parametrize("lengths", LENGTHS, ids=[f"len{i}" for i in range(len(LENGTHS))])
def test_lengths_and_masks(lengths, pattern, D):
    go(Case(*lengths, D=D, seed=len(lengths[0])), pattern)


@pytest.mark.parametrize("page", [16, 32, 64, 128, 256])
@pytest.mark.parametrize("token_major", [False, True])
@pytest.mark.parametrize("heads", [(1, 1), (3, 3), (8, 1), (12, 4), (5, 1), (16, 2), (33, 1), (40, 1)])
def test_pages_and_heads(page, token_major, heads):
    Hq, Hkv = heads
    go(Case([1, 2, 1], [77, 600, 256], Hq=Hq, Hkv=Hkv, D=64, page=page, token_major=token_major, seed=page), WS)
    go(Case([1, 90], [1000, 300], Hq=Hq, Hkv=Hkv, D=128, page=page, token_major=token_major, seed=page + 1), ALL)


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("prefix", [1, 16, 100, 1000, 2043])
@pytest.mark.parametrize("lengths", [([1] * 6, [1, 2, 30, 64, 65, 200]), ([1, 0, 7, 1], [5, 3, 7, 0]),
                                     ([1] * 40, list(range(1, 41))), ([150, 1], [300, 20])],
                         ids=["ones", "ragged", "many", "piece"])
def test_shared_prefix(lengths, prefix, D):
    go(Case(*lengths, D=D, prefix=prefix, Hq=8, Hkv=2, page=32, seed=prefix), ALL)
    go(Case(*lengths, D=D, prefix=prefix, Hq=4, Hkv=4, page=16, seed=prefix, token_major=True), WS)


def test_shared_prefix_equals_one_cache():
    """A prefix held apart gives what the whole sequences in one cache give."""
    c = Case([1, 3, 2], [9, 40, 77], prefix=130, Hq=4, Hkv=2, D=64, page=16, seed=5)
    w = Case([1, 3, 2], [139, 170, 207], Hq=4, Hkv=2, D=64, page=16, seed=6)
    w.q, w.k, w.v = c.q, c.k, c.v
    for b in range(3):
        n = -(-w.kv_len[b] // 16)
        w._put(w.table[b, :n].tolist(), c.k[b], c.v[b])
    for p in (ALL, WS, sa.Pattern(window=20, sinks=7)):
        (o1, l1), (o2, l2) = c.run(p), w.run(p)
        c.check(o2, l2, p)
        c.check(o1, l1, p)


@pytest.mark.parametrize("max_q", [0, 1, 64, 4096])
def test_max_q_is_a_hint(max_q):
    c = Case([1, 50, 300], [200, 90, 700], seed=3)
    o, lse = c.run(WS, max_q=max_q)
    c.check(o, lse, WS)


def test_many_sequences():
    B = 700
    kv = [1 + (37 * b) % 211 for b in range(B)]
    go(Case([1] * B, kv, Hq=4, Hkv=2, D=64, seed=11), ALL)
    q = [(b * 7) % 3 for b in range(B)]
    go(Case(q, [n + m for n, m in zip(kv, q)], Hq=2, Hkv=2, D=64, seed=12), WS)


def test_long_cache():
    go(Case([1, 1], [40000, 3], Hq=8, Hkv=1, D=128, page=64, seed=21), ALL)
    go(Case([1], [30001], Hq=2, Hkv=2, D=64, page=16, seed=22), sa.Pattern(window=5000, sinks=130))
    go(Case([600], [9000], Hq=4, Hkv=1, D=128, page=64, seed=23), sa.Pattern(window=3000, sinks=4))
    go(Case([1] * 70, [3] * 70, Hq=8, Hkv=2, D=128, page=64, prefix=12000, seed=24), ALL)


def test_large_scores_and_scale():
    c = Case([1, 3, 150], [500, 80, 400], seed=31, q_scale=8.0)
    go(c, ALL)
    go(c, WS, scale=0.5)


def test_strided_queries_and_outputs_rows_behind_the_last():
    c = Case([1, 4, 33], [90, 200, 33], pad_rows=5, seed=41)
    wide = torch.full((c.T, c.Hq + 3, c.D), 7.0, dtype=torch.bfloat16, device="cuda")
    wide[:, 2:2 + c.Hq] = c.dev(c.q)
    out = torch.full((c.Hq, c.T, c.D), 3.0, dtype=torch.bfloat16, device="cuda").transpose(0, 1)
    lse = torch.full((c.T, c.Hq), 5.0, device="cuda")
    o, l = sa.fwd_cached(wide[:, 2:2 + c.Hq], c.cache(), c.batch(33), WS, out=out, lse=lse)
    assert o.data_ptr() == out.data_ptr()
    c.check(o, l, WS)
    T = int(c.q_start[-1])
    assert bool((out[T:] == 3).all()) and bool((lse[T:] == 5).all())


def test_bit_identical_and_other_streams():
    c = Case([1] * 9 + [140], [3000, 1, 40, 77, 600, 5000, 2, 64, 128, 900], Hq=8, Hkv=2, seed=51)
    o, l = c.run(ALL)
    q, cache, batch = c.dev(c.q), c.cache(), c.batch(140)
    torch.cuda.synchronize()
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    got = []
    for _ in range(5):  # two streams at once, a workspace each
        for s in (s1, s2):
            got.append(sa.fwd_cached(q, cache, batch, ALL, stream=s))
    torch.cuda.synchronize()
    for a, b in got:
        assert torch.equal(a, o) and torch.equal(b, l)


def test_captured_graph_follows_lengths():
    """A captured step replayed with other lengths and tables."""
    c = Case([1] * 4, [100, 7, 64, 300], Hq=8, Hkv=2, page=16, seed=61)
    d = Case([1] * 4, [3, 200, 310, 1], Hq=8, Hkv=2, page=16, seed=62)
    width = max(c.table.shape[1], d.table.shape[1])
    n = max(c.k_pages.shape[0], d.k_pages.shape[0])
    k, v = (torch.zeros((n,) + tuple(c.k_pages.shape[1:]), dtype=torch.bfloat16, device="cuda") for _ in range(2))
    table = torch.full((4, width), -1, dtype=torch.int32, device="cuda")
    kv_len = torch.zeros(4, dtype=torch.int32, device="cuda")
    q = torch.zeros(c.T, c.Hq, c.D, dtype=torch.bfloat16, device="cuda")
    cache, batch = sa.KVCache(k, v), sa.CacheBatch(c.dev(c.q_start), kv_len, table, max_q=1)

    def load(x):
        k[:x.k_pages.shape[0]].copy_(x.k_pages)
        v[:x.v_pages.shape[0]].copy_(x.v_pages)
        table[:, :x.table.shape[1]].copy_(x.table)
        kv_len.copy_(torch.tensor(x.kv_len, dtype=torch.int32))
        q.copy_(x.q)

    load(c)
    sa.fwd_cached(q, cache, batch, ALL)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        o, l = sa.fwd_cached(q, cache, batch, ALL)
    for x in (c, d, c):
        load(x)
        g.replay()
        torch.cuda.synchronize()
        x.check(o, l, ALL)


def test_bad_pages_read_as_zeros():
    """A page outside the cache holds keys and values of zero; the first 32 tokens sit on one here."""
    c = Case([1, 1], [90, 40], Hq=2, Hkv=1, D=64, page=32, seed=71)
    c.table[0, 0] = c.k_pages.shape[0]
    c.table[1, 0] = -1
    for b in range(2):
        c.k[b][:32] = 0
        c.v[b][:32] = 0
    go(c, ALL)


def test_lengths_beyond_the_table_and_negative():
    c = Case([1, 2, 1], [40, 3, 20], Hq=2, Hkv=1, D=64, page=16, seed=81)
    kv = torch.tensor([40, -5, 20], dtype=torch.int32, device="cuda")
    batch = sa.CacheBatch(c.dev(c.q_start), kv, c.dev(c.table), max_q=2)
    o, l = sa.fwd_cached(c.dev(c.q), c.cache(), batch, ALL)
    c.kv_len = [40, 0, 20]
    c.k[1], c.v[1] = c.k[1][:0], c.v[1][:0]
    c.check(o, l, ALL)
    kv[0] = 10 ** 6  # read as the table's room: 48 or more places, the last ones on bad pages
    sa.fwd_cached(c.dev(c.q), c.cache(), batch, ALL)
    assert sa.check_device() == sa.SA_OK


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("q_len,group", [(1, 4), (1, 6), (3, 8)])
def test_ragged_batches_cut_over_the_ctas(q_len, group, D):
    """Long and short sequences in one batch: items cut by several CTAs, items of one unit between them."""
    kv = [q_len + (9000 * b * b // 1600) % 9001 for b in range(40)]
    go(Case([q_len] * 40, kv, Hq=2 * group, Hkv=2, D=D, page=32, seed=101), ALL)
    go(Case([q_len] * 40, kv, Hq=2 * group, Hkv=2, D=D, page=16, seed=102), sa.Pattern(window=3000, sinks=70))


def test_more_items_than_clusters():
    """Whole items by clusters of CTAs, several items one after another."""
    kv = [3 + (41 * b) % 300 for b in range(90)]
    go(Case([1] * 90, kv, Hq=8, Hkv=4, D=128, seed=103), sa.Pattern(window=60, sinks=4))
    go(Case([2] * 150, [n + 2 for n in kv] + [5] * 60, Hq=16, Hkv=4, D=64, seed=104), sa.Pattern(window=40, sinks=1))
    for heads in (1, 2, 5, 9, 18, 40):  # clusters of eight, four, two, one
        go(Case([1], [1500], Hq=heads, Hkv=heads, D=64, seed=heads), sa.Pattern(window=900, sinks=2))


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("prefix", [0, 500])
@pytest.mark.parametrize("q_len,Hq,Hkv,kv_max", [(1, 8, 4, 600), (1, 16, 8, 30), (4, 8, 2, 300), (2, 40, 5, 900),
                                                 (1, 7, 7, 17)])
def test_short_sequences_cut_over_the_warps(q_len, Hq, Hkv, kv_max, prefix, D):
    """An item or more to every CTA and few keys to each; empty sequences and lengths of one among them."""
    B = -(-600 // Hkv) + 37
    m = [q_len if b % 11 else b % 2 for b in range(B)]
    kv = [max(n, 1 + (53 * b) % kv_max) if b % 13 else n for b, n in enumerate(m)]
    go(Case(m, kv, Hq=Hq, Hkv=Hkv, D=D, page=16, prefix=prefix, seed=111), ALL)
    go(Case(m, kv, Hq=Hq, Hkv=Hkv, D=D, page=64, prefix=prefix, seed=112), sa.Pattern(window=kv_max // 2, sinks=3))
    go(Case(m, kv, Hq=Hq, Hkv=Hkv, D=D, page=32, prefix=prefix, seed=113), sa.Pattern(window=-1, sinks=5))


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("prefix", [0, 300])
@pytest.mark.parametrize("q_len,Hq,Hkv", [(8, 8, 2), (5, 5, 1), (1, 17, 1), (1, 62, 2), (17, 3, 3)])
def test_seventeen_to_thirty_two_rows(q_len, Hq, Hkv, prefix, D):
    for B, far in ((3, 700), (30, 5000)):
        kv = [q_len + (31 + far * b // 7) % far for b in range(B)]
        m = [q_len - b % 2 for b in range(B)]
        go(Case(m, kv, Hq=Hq, Hkv=Hkv, D=D, prefix=prefix, seed=121), ALL)
        go(Case(m, kv, Hq=Hq, Hkv=Hkv, D=D, prefix=prefix, seed=122), sa.Pattern(window=200, sinks=40))


def test_a_warp_whose_wait_runs_out():
    """As test_a_wait_that_runs_out, where the warps of a CTA work on pieces of their own."""
    c = Case([1] * 160, [1 + (53 * b) % 200 for b in range(160)], Hq=8, Hkv=4, seed=166)
    args = (c.dev(c.q), c.cache(), c.batch(1))
    try:
        sa.set_debug(sa.DEBUG_SKIP_Q_LOAD, 20_000_000)
        sa.fwd_cached(*args, ALL)
        assert sa.check_device() == sa.SA_ERR_DEVICE_TIMEOUT
    finally:
        sa.set_debug(0, 0)
    assert sa.check_device() == sa.SA_OK
    c.check(*sa.fwd_cached(*args, ALL), ALL)


def test_short_sequences_of_graphs_sharing_a_workspace():
    """Two captured steps over one workspace, replayed in turn with other lengths of their sequences."""
    c = Case([1] * 160, [1 + (53 * b) % 400 for b in range(160)], Hq=8, Hkv=4, page=16, seed=167)
    d = Case([2] * 160, [2 + (91 * b) % 300 for b in range(160)], Hq=8, Hkv=4, page=16, seed=168)
    ws = torch.empty(max(sa.fwd_cached_workspace_bytes(x.T, x.Hq, x.Hkv, x.D) for x in (c, d)), dtype=torch.uint8,
                     device="cuda")
    steps = []
    for x in (c, d):
        args = (x.dev(x.q), x.cache(), x.batch(max(x.q_len)))
        sa.fwd_cached(*args, ALL, workspace=ws)
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            out = sa.fwd_cached(*args, ALL, workspace=ws)
        steps.append((x, g, args, out))
    for _ in range(3):
        for x, g, args, out in steps:
            g.replay()
            x.check(*out, ALL)
    for x, g, args, out in steps:
        x.kv_len = [n - (3 if n > 9 else 0) for n in x.kv_len]
        x.k, x.v = ([y[:n] for y, n in zip(z, x.kv_len)] for z in (x.k, x.v))
        args[2].kv_len.copy_(torch.tensor(x.kv_len, dtype=torch.int32))
        g.replay()
        x.check(*out, ALL)


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("q_len", [1, 3, 70, 300])
@pytest.mark.parametrize("prefix", [0, 500])
def test_infinities_in_places_no_row_sees(q_len, prefix, D):
    """Keys and values below the window of every row (and behind the sinks) are NaN and infinite."""
    p = sa.Pattern(window=100, sinks=4)
    c = Case([q_len, q_len], [1200, 1000], D=D, prefix=prefix, Hq=4, Hkv=2, page=64, seed=111)
    hidden = lambda n: (4, prefix + n - q_len - 100)  # first and last + 1 of the keys that no row sees
    for b, n in enumerate(c.kv_len):
        need = -(-n // c.page)
        lo, hi = hidden(n)
        lo, hi = max(lo - prefix, 0), hi - prefix
        k, v = c.k[b][prefix:].clone(), c.v[b][prefix:].clone()
        k[lo:hi], v[lo:hi] = math.nan, math.inf
        c._put(c.table[b, :need].tolist(), k, v)
        c.k[b], c.v[b] = c.k[b].clone(), c.v[b].clone()
        c.k[b][4:prefix + hi] = 0  # the plain form multiplies by weights of zero
        c.v[b][4:prefix + hi] = 0
    if prefix:
        k, v = torch.zeros(prefix, 2, D).bfloat16(), torch.zeros(prefix, 2, D).bfloat16()
        k[:4], v[:4] = c.k[0][:4], c.v[0][:4]
        k[4:], v[4:] = math.nan, -math.inf
        c._put(c.prefix_table.tolist(), k, v)
    go(c, p)


def test_table_shares_pages_and_fused_cache():
    """Two sequences over the same pages; keys and values in one tensor of pages."""
    c = Case([1, 1, 5], [64, 64, 100], Hq=4, Hkv=2, D=64, page=32, seed=121)
    c.table[1] = c.table[0]
    c.k[1], c.v[1] = c.k[0], c.v[0]
    both = torch.stack([c.k_pages, c.v_pages], 1).cuda()
    o, lse = sa.fwd_cached(c.dev(c.q), sa.KVCache(both[:, 0], both[:, 1]), c.batch(5), ALL)
    c.check(o, lse, ALL)


def test_no_prefix_is_the_cached_call():
    c = Case([1, 40], [700, 90], Hq=8, Hkv=2, seed=131)
    o, l = c.run(WS)
    o2, l2 = sa.fwd_shared(c.dev(c.q), c.cache(), c.batch(40), None, 0, WS)
    assert torch.equal(o, o2) and torch.equal(l, l2)


@pytest.mark.parametrize("D", [64, 128])
def test_offsets_beyond_32_bits(D):
    """Pages that lie more than 2^32 elements into the cache: attention and append."""
    c = Case([1, 150], [300, 200], Hq=2, Hkv=1, D=D, page=64, seed=141)
    n = c.k_pages.shape[0]
    total = (1 << 32) // (64 * D) + 3 * n
    k, v = (torch.empty((total, 1, 64, D), dtype=torch.bfloat16, device="cuda") for _ in range(2))
    k[-n:], v[-n:] = c.dev(c.k_pages), c.dev(c.v_pages)
    table = c.table.clone()
    for b in range(2):
        need = -(-c.kv_len[b] // 64)
        table[b, :need] += total - n
    batch = sa.CacheBatch(c.dev(c.q_start), c.dev(torch.tensor(c.kv_len, dtype=torch.int32)), c.dev(table), max_q=150)
    cache = sa.KVCache(k, v)
    o, lse = sa.fwd_cached(c.dev(c.q), cache, batch, ALL)
    c.check(o, lse, ALL)
    new = torch.randn(c.T, 1, D, device="cuda").bfloat16()
    sa.cache_append(new, new, cache, batch)
    assert torch.equal(k[int(table[0, 299 // 64]), 0, 299 % 64], new[0, 0])
    assert torch.equal(v[int(table[1, 199 // 64]), 0, 199 % 64], new[150, 0])


def test_graphs_of_pieces_and_prefixes_sharing_a_workspace():
    """Captured calls of both kernels over one workspace, replayed in turn."""
    a = Case([200, 1, 3], [900, 400, 50], Hq=8, Hkv=2, D=128, page=64, seed=151)
    b = Case([1] * 30, [9] * 30, Hq=8, Hkv=2, D=128, page=64, prefix=1500, seed=152)
    need = max(sa.fwd_cached_workspace_bytes(a.T, 8, 2, 128), sa.fwd_shared_workspace_bytes(b.T, 8, 2, 128))
    ws = torch.empty(need, dtype=torch.uint8, device="cuda")
    calls = []
    for c in (a, b):
        q, cache, batch, pt = c.dev(c.q), c.cache(), c.batch(max(c.q_len)), c.dev(c.prefix_table)
        call = (lambda q=q, cache=cache, batch=batch, pt=pt, c=c:
                sa.fwd_shared(q, cache, batch, pt, c.prefix, ALL, workspace=ws) if c.prefix else
                sa.fwd_cached(q, cache, batch, ALL, workspace=ws))
        call()
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            out = call()
        calls.append((c, g, out, call))  # the graph reads what the call holds
    for _ in range(3):
        for c, g, out, _call in calls:
            for t in out:
                t.zero_()
            g.replay()
            c.check(*out, ALL)


@pytest.mark.parametrize("kind", ["items", "line", "piece", "prefix", "prefix_many"])
def test_a_wait_that_runs_out(kind):
    """The bounded waits: a tile that is never loaded sets the status word, and the next call is sound."""
    c = {"items": lambda: Case([1] * 3, [200, 90, 30], seed=161),
         "line": lambda: Case([1] * 3, [20000, 90, 30], seed=162),
         "piece": lambda: Case([1, 300], [200, 900], seed=163),
         "prefix": lambda: Case([1] * 3, [20, 9, 3], prefix=300, seed=164),
         "prefix_many": lambda: Case([1] * 40, [20] * 40, prefix=300, seed=165)}[kind]()
    args = (c.dev(c.q), c.cache(), c.batch(max(c.q_len)))
    pt = c.dev(c.prefix_table)
    call = lambda: (sa.fwd_shared(*args, pt, c.prefix, ALL) if c.prefix else sa.fwd_cached(*args, ALL))
    try:
        sa.set_debug(sa.DEBUG_SKIP_Q_LOAD, 20_000_000)
        call()
        assert sa.check_device() == sa.SA_ERR_DEVICE_TIMEOUT
    finally:
        sa.set_debug(0, 0)
    assert sa.check_device() == sa.SA_OK  # the word was cleared
    c.check(*call(), ALL)


def test_matches_whole_sequence_attention():
    """A prompt appended to an empty cache and attended over it gives what fwd gives."""
    N, Hq, Hkv, D = 700, 4, 2, 128
    g = torch.Generator(device="cuda").manual_seed(91)
    q, k, v = (torch.randn(1, h, N, D, generator=g, device="cuda").bfloat16() for h in (Hq, Hkv, Hkv))
    p = sa.Pattern(window=200, sinks=4)
    o, lse = sa.fwd(q, k, v, sa.build_block_mask(p, N, 128).to_device("cuda"), p)
    pages = [torch.zeros(44, Hkv, 16, D, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    cache = sa.KVCache(*pages)
    table = torch.randperm(44, device="cuda").to(torch.int32)[None]
    i32 = lambda *a: torch.tensor(a, dtype=torch.int32, device="cuda")
    tok = lambda x: x[0].transpose(0, 1)
    batch = sa.CacheBatch(i32(0, N), i32(N), table, max_q=N)
    sa.cache_append(tok(k), tok(v), cache, batch)
    o2, lse2 = sa.fwd_cached(tok(q), cache, batch, p)
    # both sides within 2^-8 |O| (output) + 2^-8 max|v| (weights) of the exact value
    bound = 2 * (2.0 ** -8 * o.float().abs().max() + 2.0 ** -8 * v.float().abs().max())
    assert float((o2.transpose(0, 1)[None].float() - o.float()).abs().max()) <= float(bound)
    assert float((lse2.T[None] - lse).abs().max()) <= 2 * 1e-3


def test_serving_run():
    """Rotation, append and attention together: a prompt, then single tokens, against the whole
    sequence rotated and attended at once."""
    Hq, Hkv, D, N0, N = 4, 2, 64, 37, 45
    g = torch.Generator(device="cuda").manual_seed(95)
    B = 3
    q, k, v = (torch.randn(B, h, N, D, generator=g, device="cuda").bfloat16() for h in (Hq, Hkv, Hkv))
    spec = sa.Rotary([10000.0 ** (-i / 24) for i in range(24)])
    pos = torch.arange(N, dtype=torch.int32, device="cuda").expand(1, 1, N)
    p = sa.Pattern(window=16, sinks=2)
    qr, kr = sa.rotary(q, k, pos, spec)
    o, lse = sa.fwd(qr, kr, v, sa.build_block_mask(p, N, 128).to_device("cuda"), p)
    cache = sa.KVCache(*(torch.full((16, Hkv, 16, D), math.nan, dtype=torch.bfloat16, device="cuda") for _ in range(2)))
    table = torch.randperm(16, device="cuda")[:9].to(torch.int32).reshape(3, 3)
    i32 = lambda a: torch.tensor(a, dtype=torch.int32, device="cuda")
    steps = [(0, N0)] + [(i, i + 1) for i in range(N0, N)]
    for a, z in steps:
        m = z - a
        rows = lambda x: x[:, :, a:z].transpose(1, 2).reshape(B * m, x.shape[1], D)
        batch = sa.CacheBatch(i32([m * b for b in range(B + 1)]), i32([z] * B), table, max_q=m)
        qn = sa.cache_append(rows(k), rows(v), cache, batch, rotary=spec, q=rows(q))
        assert torch.equal(qn, rows(qr))
        on, ln = sa.fwd_cached(qn, cache, batch, p)
        want = o[:, :, a:z].transpose(1, 2).reshape(B * m, Hq, D)
        bound = 4 * 2.0 ** -8 * float(v.float().abs().max())  # two kernels, weights and output rounded in each
        assert float((on.float() - want.float()).abs().max()) <= bound
        assert float((ln - lse[:, :, a:z].transpose(1, 2).reshape(B * m, Hq)).abs().max()) <= 2e-3


@pytest.mark.skipif(torch.cuda.device_count() < 2, reason="needs two GPUs")
def test_other_device_than_the_current_one():
    c = Case([1, 40], [300, 90], seed=99, device="cuda:1")
    with torch.cuda.device(0):
        o, lse = sa.fwd_cached(c.dev(c.q), c.cache(), c.batch(40), WS)
    c.check(o, lse, WS)


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("q_len,Hq,Hkv,B,prefix", [(1, 8, 2, 40, 700), (2, 32, 8, 30, 151), (1, 32, 8, 6, 1500),
                                                   (3, 16, 2, 25, 1033), (1, 20, 1, 9, 90), (8, 8, 2, 2, 640)])
def test_parts_of_a_prefix_added_by_the_sequences_pass(q_len, Hq, Hkv, B, prefix, D):
    """Few keys of its own to each sequence, behind a prefix whose items are cut into a few parts."""
    m = [q_len if b % 5 else b % 2 for b in range(B)]
    m[0] = q_len
    kv = [max(n, (37 * b) % 130) for b, n in enumerate(m)]
    for page, pattern in ((32, ALL), (64, sa.Pattern(window=120, sinks=70)), (16, sa.Pattern(window=-1, sinks=300))):
        c = Case(m, kv, Hq=Hq, Hkv=Hkv, D=D, page=page, prefix=prefix, pad_rows=3, seed=171)
        o, lse = go(c, pattern)
        again, l_again = c.run(pattern)
        T = int(c.q_start[-1])
        assert torch.equal(o[:T], again[:T]) and torch.equal(lse[:T], l_again[:T])
