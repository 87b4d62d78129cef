"""GPU parity of the rotation, its backward pass and the append to a paged cache, against 64 bits."""
import math

import pytest
import torch

import block_sparse_attention_build_b200 as sa

pytestmark = pytest.mark.gpu


def plain(x, pos, freq, axis, interleaved, sign=1.0):
    """x [..., D] in 64 bits, pos [axes, ...] broadcast over x's leading dimensions."""
    P = len(freq)
    x = x.double()
    ang = torch.stack([pos[a].double() * f for a, f in zip(axis, freq)], -1) * sign if P else x[..., :0]
    c, s = torch.cos(ang), torch.sin(ang)
    y = x.clone()
    ia = torch.arange(P) * 2 if interleaved else torch.arange(P)
    ib = ia + 1 if interleaved else ia + P
    y[..., ia] = x[..., ia] * c - x[..., ib] * s
    y[..., ib] = x[..., ib] * c + x[..., ia] * s
    size = x.abs()
    size[..., ia] = size[..., ib] = x[..., ia].abs() + x[..., ib].abs()
    return y, size


def check(got, x, *args):
    """Sine and cosine are within 2^-21 (the angle's rounding to 32 bits, 2^-24 pi, and the function's
    last places), the two products and their sum within 2^-23; the result is rounded once, 2^-8."""
    y, size = plain(x, *args)
    over = (got.double() - y).abs() - (2.0 ** -8 * y.abs() * (1 + 2.0 ** -12) + 2.0 ** -20 * size)
    assert bool((over <= 0).all()), float(over.max())
    P = len(args[1])
    assert torch.equal(got[..., 2 * P:], x[..., 2 * P:])


def spec_of(P, axes, interleaved):
    freq = [10000.0 ** (-i / max(P, 1)) for i in range(P)]
    axis = [(i * axes) // max(P, 1) for i in range(P)]
    return freq, axis, sa.Rotary(freq, axis=axis, interleaved=interleaved, n_axes=axes)


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("D,P,axes", [(128, 64, 1), (128, 62, 3), (128, 47, 2), (128, 56, 4), (64, 32, 2), (64, 30, 3),
                                      (64, 15, 1), (64, 24, 3), (64, 1, 1), (64, 0, 1), (128, 8, 1)])
def test_rotary(D, P, axes, interleaved):
    freq, axis, spec = spec_of(P, axes, interleaved)
    g = torch.Generator(device="cuda").manual_seed(P)
    for B, Hq, Hkv, N in [(1, 1, 1, 1), (2, 6, 2, 77), (3, 9, 0, 40), (1, 33, 4, 130)]:
        q = torch.randn(B, Hq, N, D, generator=g, device="cuda").bfloat16()
        k = torch.randn(B, Hkv, N, D, generator=g, device="cuda").bfloat16() if Hkv else None
        pos = torch.randint(-50, 300000, (axes, B, N), generator=g, device="cuda", dtype=torch.int32)
        for fn, sign in ((sa.rotary, 1.0), (sa.rotary_bwd, -1.0)):
            for x, y in zip((q, k), fn(q, k, pos, spec)):
                if x is None:
                    assert y is None
                    continue
                check(y, x, pos[:, :, None], freq, axis, interleaved, sign)


def test_rotary_strides_broadcast_positions_and_in_place():
    freq, axis, spec = spec_of(60, 2, False)
    B, N, Hq, Hkv, D = 2, 50, 5, 3, 128
    x = torch.randn(B, N, Hq + 2 * Hkv, D, device="cuda").bfloat16()
    keep = x.clone()
    q, k = x[:, :, :Hq].transpose(1, 2), x[:, :, Hq:Hq + Hkv].transpose(1, 2)
    pos = torch.randint(0, 5000, (2, 1, N), device="cuda", dtype=torch.int32)
    a, b = sa.rotary(q, k, pos, spec)
    check(a, q, pos[:, :, None], freq, axis, False)
    check(b, k, pos[:, :, None], freq, axis, False)
    a2, b2 = sa.rotary(q, k, pos, spec, q_out=q, k_out=k)
    assert a2.data_ptr() == q.data_ptr() and torch.equal(a2, a) and torch.equal(b2, b)
    assert torch.equal(x[:, :, Hq + Hkv:], keep[:, :, Hq + Hkv:])


def test_rotary_far_positions_and_values_it_keeps():
    freq, axis, spec = spec_of(24, 1, True)
    q = torch.randn(1, 2, 4, 64, device="cuda").bfloat16()
    q[0, 0, 0, 48:] = torch.tensor([math.nan, math.inf, -math.inf, -0.0] * 4, device="cuda").bfloat16()
    pos = torch.tensor([2 ** 31 - 1, -2 ** 31, 10 ** 8 + 7, 0], dtype=torch.int32, device="cuda").expand(1, 1, 4)
    y, _ = sa.rotary(q, None, pos.contiguous(), spec)
    assert torch.equal(y[..., 48:].view(torch.int16), q[..., 48:].view(torch.int16))
    z, size = plain(q[..., :48], pos[:, :, None], freq, axis, True)
    # 64-bit angles of 2^31 radians: 2^-21 more on either side
    assert bool(((y[..., :48].double() - z).abs() <= 2.0 ** -8 * z.abs() + 2.0 ** -19 * size).all())


def test_rotary_frequencies_of_any_size():
    """Negative frequencies, whole and many turns a position, and none."""
    freq = [-1.0, 2 * math.pi, -2 * math.pi, 100.0, -12345.678, 1e9, 0.0, 1e-12]
    spec = sa.Rotary(freq)
    q = torch.randn(1, 3, 5, 64, device="cuda").bfloat16()
    pos = torch.tensor([0, 1, -3, 77, 12], dtype=torch.int32, device="cuda").expand(1, 1, 5).contiguous()
    y, _ = sa.rotary(q, None, pos, spec)
    z, size = plain(q, pos[:, :, None], freq, [0] * 8, False)
    # both sides reduce 1e9 x 77 radians from 64 bits: 2^-53 of that, 2^-17 radians
    assert bool(((y.double() - z).abs() <= 2.0 ** -8 * z.abs() + 2.0 ** -15 * size).all())


def test_rotary_gradient_against_differences():
    """<R x, y> differentiates to R^T y: the backward call against differences of the forward in 64 bits."""
    freq, axis, spec = spec_of(30, 3, False)
    g = torch.Generator(device="cuda").manual_seed(5)
    x = torch.randn(1, 2, 3, 64, generator=g, device="cuda").bfloat16()
    dy = torch.randn(1, 2, 3, 64, generator=g, device="cuda").bfloat16()
    pos = torch.randint(0, 900, (3, 1, 3), generator=g, device="cuda", dtype=torch.int32)
    dx, none = sa.rotary_bwd(dy, None, pos, spec)
    assert none is None
    f = lambda z: float((plain(z, pos[:, :, None], freq, axis, False)[0] * dy.double()).sum())
    size = plain(dy, pos[:, :, None], freq, axis, False)[1]
    for e in range(64):
        z = x.double().clone()
        z[0, 1, 2, e] += 0.5
        up = f(z)
        z[0, 1, 2, e] -= 1.0
        diff = up - f(z)
        assert abs(float(dx[0, 1, 2, e]) - diff) <= 2.0 ** -8 * abs(diff) + 2.0 ** -19 * float(size[0, 1, 2, e]) + 1e-9


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("token_major", [False, True])
@pytest.mark.parametrize("D,P,axes", [(128, 64, 1), (64, 30, 3), (128, 47, 2)])
@pytest.mark.parametrize("q_len,kv_len", [([1], [1]), ([1] * 9, [1, 16, 17, 200, 31, 32, 33, 5, 64]),
                                          ([0, 3, 0, 0, 40, 1, 0], [0, 20, 7, 0, 40, 300, 0]),
                                          ([1] * 100, [3 + b for b in range(100)])])
def test_append(q_len, kv_len, D, P, axes, token_major, interleaved):
    freq, axis, spec = spec_of(P, axes, interleaved)
    B, T, Hq, Hkv, page = len(q_len), sum(q_len) + 3, 6, 2, 16
    g = torch.Generator(device="cuda").manual_seed(T)
    need = [-(-n // page) for n in kv_len]
    n_pages = sum(need) + 2
    shape = (n_pages, page, Hkv, D) if token_major else (n_pages, Hkv, page, D)
    pages = [torch.randn(shape, generator=g, device="cuda").bfloat16() for _ in range(2)]
    pages = [x.transpose(1, 2) if token_major else x for x in pages]
    old = [x.clone() for x in pages]
    order = torch.randperm(n_pages, generator=g, device="cuda").to(torch.int32)
    table = torch.full((B, max(need) + 1), -1, dtype=torch.int32, device="cuda")
    at = 0
    for b in range(B):
        table[b, :need[b]] = order[at:at + need[b]]
        at += need[b]
    x = torch.randn(T, Hq + 2 * Hkv, D, generator=g, device="cuda").bfloat16()
    q, k, v = x[:, :Hq], x[:, Hq:Hq + Hkv], x[:, Hq + Hkv:]
    i32 = lambda a: torch.tensor(a, dtype=torch.int32, device="cuda")
    start = [sum(q_len[:b]) for b in range(B + 1)]
    cache, batch = sa.KVCache(*pages), sa.CacheBatch(i32(start), i32(kv_len), table)
    pos = torch.randint(0, 4000, (axes, T), generator=g, device="cuda", dtype=torch.int32)
    q_out = torch.full((T, Hq, D), 9.0, dtype=torch.bfloat16, device="cuda")
    place = torch.tensor([n - m + i for m, n in zip(q_len, kv_len) for i in range(m)], device="cuda", dtype=torch.int32)
    R = start[-1]
    for positions, where, offset in ((pos, pos[:, :R], 0), (None, (place + 5).expand(axes, R), 5)):
        for p_, o_ in zip(pages, old):
            p_.copy_(o_)
        got = sa.cache_append(k, v, cache, batch, rotary=spec, positions=positions, pos_offset=offset, q=q, q_out=q_out)
        check(got[:R], q[:R], where[:, :, None], freq, axis, interleaved)
        assert bool((q_out[R:] == 9).all())
        want_k, want_v = old[0].clone(), old[1].clone()
        t = 0
        for b in range(B):
            for i in range(q_len[b]):
                s = kv_len[b] - q_len[b] + i
                pg = int(table[b, s // page])
                check(pages[0][pg, :, s % page], k[t], where[:, t][:, None], freq, axis, interleaved)
                want_k[pg, :, s % page] = pages[0][pg, :, s % page]
                want_v[pg, :, s % page] = v[t]
                t += 1
        assert torch.equal(pages[0], want_k) and torch.equal(pages[1], want_v)
    # without a rotation: a copy
    sa.cache_append(k, v, cache, batch)
    t = 0
    for b in range(B):
        for i in range(q_len[b]):
            s = kv_len[b] - q_len[b] + i
            assert torch.equal(pages[0][int(table[b, s // page]), :, s % page], k[t])
            t += 1


def test_append_drops_what_has_no_place():
    """Places before 0, behind the table or on a page outside the cache are not written."""
    pages = [torch.zeros(3, 1, 16, 64, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    i32 = lambda a: torch.tensor(a, dtype=torch.int32, device="cuda")
    # sequence 0: places -2 .. 1; 1: 31 .. 32 (the table ends at 32); 2: on page 3; 3: on page -1
    batch = sa.CacheBatch(i32([0, 4, 6, 7, 8]), i32([2, 33, 1, 1]), i32([[0, 0], [1, 2], [3, 0], [-1, 0]]))
    k = torch.arange(1, 9, device="cuda").bfloat16()[:, None, None].expand(8, 1, 64).contiguous()
    sa.cache_append(k, k, sa.KVCache(*pages), batch)
    want = torch.zeros_like(pages[0])
    want[0, 0, 0], want[0, 0, 1], want[2, 0, 15] = 3, 4, 5
    assert torch.equal(pages[0], want) and torch.equal(pages[1], want)
