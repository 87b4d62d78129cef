"""Rotation and append of many tokens and heads: threads that own many heads, whole batches of loads with a
rest, blocks in several rounds."""
import pytest
import torch

import block_sparse_attention_build_b200 as sa
from test_rotary_gpu import check, spec_of

pytestmark = pytest.mark.gpu


def heads_per(rows, heads, D, P, interleaved):
    """Heads of one thread, as the launch chooses them on the current device."""
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    shuffled = not interleaved and P % 8 != 0
    blocks = -(-rows * (D // (4 if shuffled else 16)) // 128)
    held = (8 if shuffled else 6) * sms
    few = 3 * blocks <= 2 * held
    parts = max(held // blocks, 3) if few else -(-3 * held // blocks)
    per = -(-heads // parts)
    return -(-max(per, 0 if few else 16) // 4) * 4, few


# (D, P, axes, interleaved, B, N, Hq, Hkv, heads of a thread): every layout, few and many blocks
SHAPES = [(64, 30, 3, False, 2, 20000, 8, 1, 16), (64, 30, 3, False, 2, 16384, 64, 8, 24),
          (64, 15, 1, False, 1, 40000, 11, 2, 16), (128, 47, 2, False, 1, 9000, 21, 5, 16),
          (128, 64, 1, False, 1, 9999, 19, 2, 16), (128, 64, 2, True, 3, 7000, 37, 6, 16),
          (64, 32, 1, True, 1, 30011, 33, 3, 16), (64, 24, 2, False, 2, 12001, 30, 7, 16),
          (128, 62, 1, False, 1, 3000, 45, 9, 20), (128, 61, 1, False, 1, 5001, 45, 9, 20)]


@pytest.mark.parametrize("D,P,axes,interleaved,B,N,Hq,Hkv,per", SHAPES)
def test_rotary_of_many_tokens(D, P, axes, interleaved, B, N, Hq, Hkv, per):
    freq, axis, spec = spec_of(P, axes, interleaved)
    assert heads_per(B * N, Hq + Hkv, D, P, interleaved)[0] >= min(per, 8)  # more than the small calls' four
    g = torch.Generator(device="cuda").manual_seed(P)
    x = torch.randn(B, N, Hq + 2 * Hkv, D, generator=g, device="cuda").bfloat16()
    keep = x.clone()
    q, k = x[:, :, :Hq].transpose(1, 2), x[:, :, Hq:Hq + Hkv].transpose(1, 2)
    pos = torch.randint(0, 20000, (axes, B, N), generator=g, device="cuda", dtype=torch.int32)
    for fn, sign in ((sa.rotary, 1.0), (sa.rotary_bwd, -1.0)):
        for got, was in zip(fn(q, k, pos, spec), (q, k)):
            for h in range(0, got.shape[1], 8):  # in 64 bits, a few heads at a time
                check(got[:, h:h + 8], was[:, h:h + 8], pos[:, :, None], freq, axis, interleaved, sign)
    a, b = sa.rotary(q, k, pos, spec)
    sa.rotary(q, k, pos, spec, q_out=q, k_out=k)
    assert torch.equal(q, a) and torch.equal(k, b)
    assert torch.equal(x[:, :, Hq + Hkv:], keep[:, :, Hq + Hkv:])


@pytest.mark.parametrize("token_major", [False, True])
@pytest.mark.parametrize("D,P,axes,interleaved", [(64, 30, 3, False), (64, 32, 1, False), (128, 47, 1, False),
                                                  (128, 64, 1, True), (64, 15, 2, False)])
def test_append_of_many_tokens(D, P, axes, interleaved, token_major):
    """Threads that go from queries to keys to values, with whole batches of heads and a rest in each."""
    freq, axis, spec = spec_of(P, axes, interleaved)
    Hq, Hkv, page = 26, 11, 64
    q_len = [5000, 1, 0, 2999, 37]
    kv_len = [n + 77 * b for b, n in enumerate(q_len)]
    T, R = sum(q_len) + 9, sum(q_len)
    assert heads_per(T, Hq + 2 * Hkv, D, P, interleaved)[0] >= 8
    need = [-(-n // page) for n in kv_len]
    n_pages = sum(need) + 2
    g = torch.Generator(device="cuda").manual_seed(T + P)
    shape = (n_pages, page, Hkv, D) if token_major else (n_pages, Hkv, page, D)
    pages = [torch.randn(shape, generator=g, device="cuda").bfloat16() for _ in range(2)]
    pages = [x.transpose(1, 2) if token_major else x for x in pages]
    old = [x.clone() for x in pages]
    order = torch.randperm(n_pages, generator=g, device="cuda").to(torch.int32)
    table = torch.full((len(q_len), max(need)), -1, dtype=torch.int32, device="cuda")
    at = 0
    for b, n in enumerate(need):
        table[b, :n] = order[at:at + n]
        at += n
    i32 = lambda a: torch.tensor(a, dtype=torch.int32, device="cuda")
    start = [sum(q_len[:b]) for b in range(len(q_len) + 1)]
    x = torch.randn(T, Hq + 2 * Hkv, D, generator=g, device="cuda").bfloat16()
    q, k, v = x[:, :Hq], x[:, Hq:Hq + Hkv], x[:, Hq + Hkv:]
    q_out = torch.full((T, Hq, D), 9.0, dtype=torch.bfloat16, device="cuda")
    place = i32([n - m + i for m, n in zip(q_len, kv_len) for i in range(m)]).long()
    seq = torch.repeat_interleave(torch.arange(len(q_len), device="cuda"), i32(q_len))
    pos = place.int().expand(axes, R)
    sa.cache_append(k, v, sa.KVCache(*pages), sa.CacheBatch(i32(start), i32(kv_len), table), rotary=spec, q=q,
                    q_out=q_out)
    check(q_out[:R], q[:R], pos[:, :, None], freq, axis, interleaved)
    assert bool((q_out[R:] == 9).all())
    pg, slot = table[seq, place // page].long(), place % page
    check(pages[0][pg, :, slot], k[:R], pos[:, :, None], freq, axis, interleaved)
    assert torch.equal(pages[1][pg, :, slot], v[:R])
    for new, was in zip(pages, old):  # and nothing else was written
        was[pg, :, slot] = new[pg, :, slot]
        assert torch.equal(new, was)
