"""Cases of the cached-attention and rotary operators, with their plain forms.

A case names one of four operators:

  rotary   rotation of queries and keys by positions with one to three axes, before the
           attention of a training step, and its backward pass;
  append   new keys and values of a batch written to a paged cache, keys and queries rotated;
  cached   attention of new queries over a paged cache under a causal window and sinks;
  shared   the same for a batch whose sequences begin with one common prefix.

``run`` computes a case with elementary torch operations, or, where ``own`` is set, with the
package's operators on the same state.  Rows, heads and pages are laid out as a serving loop has
them: tokens of all sequences one after another, a page table per sequence.
"""
import math

import torch

own = False

DEV = "cuda"


def listed():
    return [
        # queries and keys of the pages' own example, read in place from a fused projection's output
        dict(name="rotary_fwd_n8192", op="rotary", B=1, Hq=16, Hkv=16, N=8192, D=128, axes=1, pairs=64,
             interleaved=False, fused=True, backward=False),
        # one 40 x 40 feature map, row and column as two axes: a small call
        dict(name="rotary_image_n1600", op="rotary", B=1, Hq=8, Hkv=8, N=1600, D=64, axes=2, pairs=32,
             interleaved=True, fused=False, backward=False),
        # time, height and width of two videos, many heads: the gradient's way back through the rotation
        dict(name="rotary_video_bwd_n16384", op="rotary", B=2, Hq=64, Hkv=8, N=16384, D=64, axes=3, pairs=30,
             interleaved=False, fused=False, backward=True),
        # one decoding step of 64 sequences: a call of a few microseconds
        dict(name="append_step_b64", op="append", B=64, Hq=32, Hkv=8, D=128, page=16, q_len=1, kv_max=32768,
             pairs=64, axes=1, interleaved=False, token_major=False),
        # prompts of several sequences, image positions, pages that keep a token's heads together
        dict(name="append_prompts_16k", op="append", B=9, Hq=64, Hkv=8, D=64, page=64, q_len=1829, kv_max=4096,
             pairs=32, axes=3, interleaved=False, token_major=True),
        # one sequence, one token, a window and four sinks: latency
        dict(name="cached_one_w1024_s4", op="cached", B=1, Hq=16, Hkv=16, D=128, page=64, q_len=1, kv_max=8192,
             window=1024, sinks=4, token_major=False),
        # a serving batch of very different lengths that sees everything, grouped heads, small pages
        dict(name="cached_batch_b64", op="cached", B=64, Hq=32, Hkv=8, D=128, page=16, q_len=1, kv_max=16384,
             window=1 << 20, sinks=0, token_major=False),
        # a few tokens to check per sequence, narrow window and sinks, many heads of 64
        dict(name="cached_few_w128_s4", op="cached", B=32, Hq=64, Hkv=8, D=64, page=32, q_len=4, kv_max=16384,
             window=128, sinks=4, token_major=True),
        # pieces of long prompts under a long window
        dict(name="cached_chunk_w4096", op="cached", B=3, Hq=32, Hkv=8, D=128, page=64, q_len=2048, kv_max=32768,
             window=4096, sinks=4, token_major=False),
        # a piece of one long prompt that sees all before it: the largest amount of arithmetic
        dict(name="cached_prompt_32k", op="cached", B=1, Hq=32, Hkv=8, D=128, page=128, q_len=4096, kv_max=32768,
             window=1 << 20, sinks=0, token_major=False),
        # a few answers to one question: short prefix, single tokens, no grouped heads
        dict(name="shared_small_b8", op="shared", B=8, Hq=16, Hkv=16, D=128, page=64, q_len=1, kv_max=128,
             prefix=2043, window=1 << 20, sinks=0, token_major=False),
        # many sequences behind one long document
        dict(name="shared_b64_32k", op="shared", B=64, Hq=32, Hkv=8, D=128, page=64, q_len=1, kv_max=1024,
             prefix=32768, window=1 << 20, sinks=0, token_major=False),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["rotary", "append", "cached", "cached", "shared"])
    Hkv = rng.choice([1, 2, 4, 8, 16])
    group = rng.choice([1, 2, 3, 4, 6, 8]) if Hkv <= 8 else rng.choice([1, 2])
    c = dict(op=op, Hq=Hkv * group, Hkv=Hkv, D=rng.choice([64, 128]))
    if op == "rotary":
        c["B"] = rng.choice([1, 2, 3, 4])
        c["N"] = _log(rng, 1, 16384 // c["B"])
    else:
        c["page"] = rng.choice([16, 32, 64, 128])
        c["token_major"] = rng.random() < 0.4
    if op in ("rotary", "append"):
        c["axes"] = rng.choice([1, 2, 3])
        c["pairs"] = c["D"] // 2 - rng.choice([0, 0, 2, 8, 17])
        c["interleaved"] = rng.random() < 0.5
    if op == "rotary":
        c["fused"] = rng.random() < 0.5
        c["backward"] = rng.random() < 0.5
        return c
    if op == "append":
        c["B"] = _log(rng, 1, 128)
        c["q_len"] = rng.choice([1, 1, _log(rng, 2, max(2, 12288 // c["B"]))])
        c["kv_max"] = c["q_len"] + _log(rng, 1, 8192)
        return c
    c["window"] = rng.choice([1 << 20, 1 << 20, _log(rng, 1, 8192)])
    c["sinks"] = rng.choice([0, 0, 4, _log(rng, 1, 300)])
    if op == "shared":
        c["B"] = _log(rng, 2, 100)
        c["q_len"] = rng.choice([1, 1, 1, _log(rng, 2, 16)])
        c["prefix"] = _log(rng, 100, 32768)
        c["kv_max"] = c["q_len"] + _log(rng, 1, 1024)
        return c
    if rng.random() < 0.6:  # decoding, one or a few tokens a sequence
        c["B"] = _log(rng, 1, 96)
        c["q_len"] = rng.choice([1, 1, 1, _log(rng, 2, 16)])
        c["kv_max"] = c["q_len"] + _log(rng, 1, min(32768, 600000 // c["B"]))
    else:  # prompts and pieces of them
        c["B"] = _log(rng, 1, 6)
        c["q_len"] = _log(rng, 17, 3000 // c["B"])
        c["kv_max"] = c["q_len"] + _log(rng, 1, 24000)
    return c


# ---------------------------------------------------------------------------- inputs

def _lengths(c):
    """Tokens of every sequence: new ones and cached ones (the new ones among them).  Fixed by the
    case: the first sequence is the longest, the others spread down to a thirtieth of it."""
    B, q_max, kv_max = c["B"], c["q_len"], c["kv_max"]
    q, kv = [], []
    for b in range(B):
        f = 30.0 ** (-((b * 0.6180339887) % 1.0)) if b else 1.0
        g = 1.0 - ((b * 0.3819660113) % 1.0) * 0.5 if b else 1.0
        n = max(1, int(q_max * g))
        q.append(n)
        kv.append(n + int((kv_max - q_max) * f))
    return q, kv


def _normal(shape, gen):
    out = torch.empty(shape, dtype=torch.bfloat16, device=DEV)
    return out.normal_(generator=gen)


def _freqs(c):
    """Rotation frequencies (radians a position) and axis of each of the case's pairs."""
    P, A = c["pairs"], c["axes"]
    per = -(-P // A)
    if A == 1:
        return [10000.0 ** (-i / P) for i in range(P)], [0] * P
    return [10000.0 ** (-(i % per) / per) for i in range(P)], [i // per for i in range(P)]


def _positions(c, first, n):
    """Positions [axes, n] of n tokens from `first` on; a grid for two and three axes."""
    t = torch.arange(first, first + n, dtype=torch.int64)
    if c["axes"] == 1:
        p = [t]
    elif c["axes"] == 2:
        p = [t // 40, t % 40]
    else:
        p = [t // 256, (t // 16) % 16, t % 16]
    return torch.stack(p).to(torch.int32)


def _paged(c, kv, gen, extra=0):
    """A cache with room for `kv` tokens a sequence (and `extra` tokens of a prefix), its page
    tables in shuffled order."""
    page, Hkv, D = c["page"], c["Hkv"], c["D"]
    need = [-(-n // page) for n in kv]
    n_extra = -(-extra // page)
    n_pages = sum(need) + n_extra + 3
    if c["token_major"]:
        k, v = (_normal((n_pages, page, Hkv, D), gen).transpose(1, 2) for _ in range(2))
    else:
        k, v = (_normal((n_pages, Hkv, page, D), gen) for _ in range(2))
    order = torch.randperm(n_pages, generator=gen, device=DEV).to(torch.int32)
    table = torch.zeros((len(kv), max(need)), dtype=torch.int32, device=DEV)
    at = 0
    for b, n in enumerate(need):
        table[b, :n] = order[at:at + n]
        at += n
    return k, v, table, order[at:at + n_extra].contiguous()


def _state(case, seed):
    c = case
    gen = torch.Generator(device=DEV)
    gen.manual_seed(seed)
    s = dict(c=c)
    if c["op"] == "rotary":
        B, Hq, Hkv, N, D = c["B"], c["Hq"], c["Hkv"], c["N"], c["D"]
        if c["fused"]:
            x = _normal((B, N, Hq + 2 * Hkv, D), gen).transpose(1, 2)
            s["q"], s["k"] = x[:, :Hq], x[:, Hq:Hq + Hkv]
        else:
            s["q"], s["k"] = _normal((B, Hq, N, D), gen), _normal((B, Hkv, N, D), gen)
        # every sequence of a batch begins somewhere else
        s["pos"] = torch.stack([_positions(c, (seed * 31 + b * 1021) % 4096, N) for b in range(B)], 1).to(DEV)
        s["freq"], s["axis"] = _freqs(c)
        return s
    q_len, kv_len = _lengths(c)
    T, Hq, Hkv, D = sum(q_len), c["Hq"], c["Hkv"], c["D"]
    s["q_len"], s["kv_len"] = q_len, kv_len
    starts = [0]
    for n in q_len:
        starts.append(starts[-1] + n)
    s["starts"] = starts
    s["k_pages"], s["v_pages"], s["table"], s["prefix_table"] = _paged(c, kv_len, gen, c.get("prefix", 0))
    s["d_start"] = torch.tensor(starts, dtype=torch.int32, device=DEV)
    s["d_len"] = torch.tensor(kv_len, dtype=torch.int32, device=DEV)
    if c["op"] == "append":
        x = _normal((T, Hq + 2 * Hkv, D), gen)
        s["q"], s["k"], s["v"] = x[:, :Hq], x[:, Hq:Hq + Hkv], x[:, Hq + Hkv:]
        s["pos"] = torch.cat([_positions(c, n - m, m) for m, n in zip(q_len, kv_len)], 1).to(DEV).contiguous()
        s["freq"], s["axis"] = _freqs(c)
    else:
        s["q"] = _normal((T, Hq, D), gen)
    return s


def prepare(case, seed):
    s = _state(case, seed)
    c = s["c"]
    if not own:
        return s
    import block_sparse_attention_build_b200 as sa
    s["sa"] = sa
    if c["op"] in ("rotary", "append"):
        s["spec"] = sa.Rotary(s["freq"], axis=s["axis"], interleaved=c["interleaved"])
    if c["op"] == "rotary":
        s["out"] = tuple(torch.empty(tuple(t.shape), dtype=t.dtype, device=DEV) for t in (s["q"], s["k"]))
        return s
    s["cache"] = sa.KVCache(s["k_pages"], s["v_pages"])
    s["batch"] = sa.CacheBatch(s["d_start"], s["d_len"], s["table"], max_q=max(s["q_len"]))
    s["out"] = torch.empty(tuple(s["q"].shape), dtype=torch.bfloat16, device=DEV)
    if c["op"] in ("cached", "shared"):
        T, Hq, D = s["q"].shape
        s["lse"] = torch.empty((T, Hq), dtype=torch.float32, device=DEV)
        s["pattern"] = sa.Pattern(window=c["window"], sinks=c["sinks"])
        need = sa.fwd_cached_workspace_bytes if c["op"] == "cached" else sa.fwd_shared_workspace_bytes
        s["workspace"] = torch.empty(need(T, Hq, c["Hkv"], D), dtype=torch.uint8, device=DEV)
    return s


# ---------------------------------------------------------------------------- plain forms

def _angles(pos, freq, axis):
    """cos, sin [..., pairs] of positions [axes, ...]: the angle in 64 bits, then 32."""
    f = torch.tensor(freq, dtype=torch.float64, device=pos.device)
    a = pos.to(torch.float64)[torch.tensor(axis, device=pos.device)]  # [pairs, ...]
    a = a.movedim(0, -1) * f
    return torch.cos(a).float(), torch.sin(a).float()


def _rotate(x, cos, sin, interleaved):
    """x [..., D]: pairs rotated by the angles (broadcast), the other elements kept."""
    P = cos.shape[-1]
    x = x.float()
    y = x.clone()
    if interleaved:
        a, b = x[..., 0:2 * P:2], x[..., 1:2 * P:2]
        y[..., 0:2 * P:2] = a * cos - b * sin
        y[..., 1:2 * P:2] = b * cos + a * sin
    else:
        a, b = x[..., :P], x[..., P:2 * P]
        y[..., :P] = a * cos - b * sin
        y[..., P:2 * P] = b * cos + a * sin
    return y.bfloat16()


def _plain_rotary(s):
    c = s["c"]
    cos, sin = _angles(s["pos"], s["freq"], s["axis"])  # [B, N, pairs]
    if c["backward"]:
        sin = -sin
    cos, sin = cos[:, None], sin[:, None]
    return [_rotate(s["q"], cos, sin, c["interleaved"]), _rotate(s["k"], cos, sin, c["interleaved"])]


def _slots(s):
    """Page and place in the page of every new token."""
    page = s["c"]["page"]
    seq = torch.repeat_interleave(torch.arange(len(s["q_len"]), device=DEV), s["d_start"].diff(),
                                  output_size=s["starts"][-1])
    T = s["starts"][-1]
    at = torch.arange(T, device=DEV) - s["d_start"][:-1][seq] + (s["d_len"] - s["d_start"].diff())[seq]
    return s["table"][seq, at // page].long(), at % page


def _plain_append(s):
    c = s["c"]
    cos, sin = _angles(s["pos"], s["freq"], s["axis"])  # [T, pairs]
    cos, sin = cos[:, None], sin[:, None]
    pg, at = _slots(s)
    s["k_pages"][pg, :, at] = _rotate(s["k"], cos, sin, c["interleaved"])
    s["v_pages"][pg, :, at] = s["v"]
    return [_rotate(s["q"], cos, sin, c["interleaved"]), s["k_pages"], s["v_pages"]]


def _gather(pages, table, n):
    """The first n tokens of a sequence's pages: [Hkv, n, D] in 32 bits."""
    page = pages.shape[2]
    x = pages[table[:-(-n // page)].long()].float()
    return x.transpose(0, 1).reshape(pages.shape[1], -1, pages.shape[3])[:, :n]


def _visible(c, p, n):
    """[len(p), n]: which of n tokens a query at position p sees."""
    kv = torch.arange(n, device=DEV)
    d = p[:, None] - kv
    return (d >= 0) & ((d <= c["window"]) | (kv < c["sinks"]))


def _plain_attention(s):
    c = s["c"]
    G, D, P = c["Hq"] // c["Hkv"], c["D"], c.get("prefix", 0)
    scale = 1.0 / math.sqrt(D)
    out = torch.empty((s["starts"][-1], c["Hq"], D), dtype=torch.bfloat16, device=DEV)
    lse = torch.empty((s["starts"][-1], c["Hq"]), dtype=torch.float32, device=DEV)
    if P:
        kp, vp = _gather(s["k_pages"], s["prefix_table"], P), _gather(s["v_pages"], s["prefix_table"], P)
    for b, (m, n) in enumerate(zip(s["q_len"], s["kv_len"])):
        t0 = s["starts"][b]
        k, v = _gather(s["k_pages"], s["table"][b], n), _gather(s["v_pages"], s["table"][b], n)
        if P:
            k, v = torch.cat([kp, k], 1), torch.cat([vp, v], 1)
        see = _visible(c, torch.arange(P + n - m, P + n, device=DEV), P + n)
        q = s["q"][t0:t0 + m].float().view(m, c["Hkv"], G, D)
        heads = range(c["Hkv"]) if m * G * (P + n) * c["Hkv"] > 1 << 27 else [slice(0, c["Hkv"])]
        for h in heads:
            h = slice(h, h + 1) if isinstance(h, int) else h
            x = torch.matmul(q[:, h].permute(1, 2, 0, 3), k[h][:, None].transpose(2, 3)) * scale  # [h, G, m, P + n]
            x = x.masked_fill(~see, -math.inf)
            top = x.amax(-1, keepdim=True)
            e = torch.exp(x - top)
            den = e.sum(-1, keepdim=True)
            o = torch.matmul(e, v[h][:, None]) / den
            hq = slice(h.start * G, h.stop * G)
            out[t0:t0 + m, hq] = o.permute(2, 0, 1, 3).reshape(m, -1, D).bfloat16()
            lse[t0:t0 + m, hq] = (top + torch.log(den))[..., 0].permute(2, 0, 1).reshape(m, -1)
    return [out, lse]


def _own(s):
    c, sa = s["c"], s["sa"]
    if c["op"] == "rotary":
        turn = sa.rotary_bwd if c["backward"] else sa.rotary
        return list(turn(s["q"], s["k"], s["pos"], s["spec"], q_out=s["out"][0], k_out=s["out"][1]))
    if c["op"] == "append":
        q = sa.cache_append(s["k"], s["v"], s["cache"], s["batch"], rotary=s["spec"], positions=s["pos"], q=s["q"],
                            q_out=s["out"])
        return [q, s["k_pages"], s["v_pages"]]
    if c["op"] == "cached":
        return list(sa.fwd_cached(s["q"], s["cache"], s["batch"], s["pattern"], out=s["out"], lse=s["lse"],
                                  workspace=s["workspace"]))
    return list(sa.fwd_shared(s["q"], s["cache"], s["batch"], s["prefix_table"], c["prefix"], s["pattern"],
                              out=s["out"], lse=s["lse"], workspace=s["workspace"]))


def run(state):
    if own:
        return _own(state)
    op = state["c"]["op"]
    if op == "rotary":
        return _plain_rotary(state)
    if op == "append":
        return _plain_append(state)
    return _plain_attention(state)


# ---------------------------------------------------------------------------- work

def _sees(c, p0, p1, P, n):
    """Visible pairs of the queries at positions p0 .. p1 - 1, and how many of the P + n tokens any
    of them sees, those of the prefix and the others apart."""
    w, sk = c["window"], c["sinks"]
    pairs = 0
    for p in range(p0, p1):
        lo = max(0, p - w)
        pairs += p + 1 - lo + min(sk, lo)
    lo = max(0, p0 - w)
    pre = max(0, P - lo) + min(sk, lo, P)
    return pairs, pre, p1 - max(lo, P) + max(0, min(sk, lo) - P)


def work(case):
    c = case
    Hq, Hkv, D = c["Hq"], c["Hkv"], c["D"]
    if c["op"] == "rotary":
        rows = c["B"] * c["N"]
        return {"bytes": 4 * rows * (Hq + Hkv) * D + 4 * rows * c["axes"], "flops": 6 * rows * (Hq + Hkv) * c["pairs"]}
    q_len, kv_len = _lengths(c)
    T = sum(q_len)
    if c["op"] == "append":
        return {"bytes": 4 * T * (Hq + 2 * Hkv) * D + 4 * T * c["axes"] + 12 * c["B"],
                "flops": 6 * T * (Hq + Hkv) * c["pairs"]}
    P = c.get("prefix", 0)
    pairs = tokens = pre = 0
    for m, n in zip(q_len, kv_len):
        a, p, t = _sees(c, P + n - m, P + n, P, n)
        pairs, pre, tokens = pairs + a, max(pre, p), tokens + t
    return {"bytes": 4 * Hkv * D * (tokens + pre) + 4 * T * Hq * D + 4 * T * Hq + 4 * (tokens + pre) // c["page"],
            "flops": 4 * pairs * Hq * D}


# ---------------------------------------------------------------------------- exact values

def _turned(x, pos, freq, axis, interleaved, sign):
    """The rotation as a product of complex numbers, 64 bits; pos [axes, ...] broadcasts over x's rows."""
    w = torch.tensor(freq, dtype=torch.float64, device=DEV)
    ang = torch.stack([pos[a].to(torch.float64) for a in axis], -1) * w * sign
    P = len(freq)
    x = x.to(torch.float64)
    head, tail = x[..., :2 * P], x[..., 2 * P:]
    re, im = (head[..., 0::2], head[..., 1::2]) if interleaved else (head[..., :P], head[..., P:])
    z = torch.complex(re.contiguous(), im.contiguous()) * torch.polar(torch.ones_like(ang), ang)
    done = torch.view_as_real(z).flatten(-2) if interleaved else torch.cat([z.real, z.imag], -1)
    return torch.cat([done, tail], -1)


def exact(case, seed):
    s = _state(case, seed)
    c = case
    if c["op"] == "rotary":
        sign = -1.0 if c["backward"] else 1.0
        pos = s["pos"][:, :, None]  # [axes, B, 1, N]
        return [_turned(s[x], pos, s["freq"], s["axis"], c["interleaved"], sign) for x in ("q", "k")]
    P = c.get("prefix", 0)
    if c["op"] == "append":
        pos = s["pos"][:, :, None]  # [axes, T, 1]
        q, k = (_turned(s[x], pos, s["freq"], s["axis"], c["interleaved"], 1.0) for x in ("q", "k"))
        kp, vp = s["k_pages"].double(), s["v_pages"].double()
        rows = s["table"].tolist()
        for b, (m, n) in enumerate(zip(s["q_len"], s["kv_len"])):
            t = s["starts"][b]
            j = n - m
            while j < n:  # the tokens of one page at a time
                pg, at = rows[b][j // c["page"]], j % c["page"]
                cnt = min(n - j, c["page"] - at)
                kp[pg, :, at:at + cnt] = k[t:t + cnt].transpose(0, 1)
                vp[pg, :, at:at + cnt] = s["v"][t:t + cnt].double().transpose(0, 1)
                t, j = t + cnt, j + cnt
        return [q, kp, vp]
    G, D = c["Hq"] // c["Hkv"], c["D"]
    out = torch.zeros((s["starts"][-1], c["Hq"], D), dtype=torch.float64, device=DEV)
    lse = torch.full((s["starts"][-1], c["Hq"]), -math.inf, dtype=torch.float64, device=DEV)
    pre = torch.arange(P, device=DEV)
    for b, (m, n) in enumerate(zip(s["q_len"], s["kv_len"])):
        t0 = s["starts"][b]
        own_at = torch.arange(n, device=DEV)
        page = torch.cat([s["prefix_table"][pre // c["page"]], s["table"][b][own_at // c["page"]]]).long()
        slot = torch.cat([pre, own_at]) % c["page"]
        p = torch.arange(m, device=DEV)[:, None] + (P + n - m)
        kv = torch.arange(P + n, device=DEV)[None, :]
        hidden = (kv > p) | ((kv < p - c["window"]) & (kv >= c["sinks"]))
        for h in range(c["Hkv"]):
            k, v = s["k_pages"][page, h, slot].double(), s["v_pages"][page, h, slot].double()
            for g in range(G):
                x = s["q"][t0:t0 + m, h * G + g].double() @ k.T / math.sqrt(D)
                x[hidden] = -math.inf
                lse[t0:t0 + m, h * G + g] = torch.logsumexp(x, -1)
                out[t0:t0 + m, h * G + g] = torch.softmax(x, -1) @ v
    return [out, lse]
