"""Order of the kernels that are set up while the stream's previous kernel still runs: by reading the
sources (CPU), and by calls whose inputs the previous call writes (GPU)."""
import os
import re

import pytest
import torch

import block_sparse_attention_build_b200 as sa
from cached_cases import Case

CSRC = os.path.join(os.path.dirname(sa.__file__), "csrc")
SOURCES = ("paged_sm100.cuh", "decode_sm100.cuh", "chunk_sm100.cuh", "rotary_sm100.cuh")


def text_of(name):
    with open(os.path.join(CSRC, name)) as f:
        return re.sub(r"//[^\n]*", "", f.read())


def kernels(text):
    """(name, body) of every __global__ function: a body ends at the first brace in the first column."""
    for m in re.finditer(r"__global__ void .*?\n\{\n(.*?)\n\}\n", text, re.S):
        yield re.search(r"(\w+_kernel)\(", m.group(0)).group(1), m.group(1)


@pytest.mark.parametrize("name", SOURCES)
def test_no_non_coherent_loads(name):
    """ld.global.nc is for data that is read-only while a kernel lives; these kernels live while the one
    before them still writes."""
    text = text_of(name)
    assert "__ldg" not in text and ".nc" not in text


def test_every_kernel_waits_before_it_touches_memory():
    seen = 0
    for name in SOURCES:
        for kernel, body in kernels(text_of(name)):
            seen += 1
            # a statement of the kernel's own block, not under a condition
            wait = body.index("\n    wait_previous_kernel();\n")
            before = body[:wait]
            assert "find_piece" not in before and "peek_seq" not in before and "load_seq" not in before, kernel
            # of the parameters, only what is passed by value (the rotation's turns) and the tensor maps
            assert not re.search(r"\bp\.", before), kernel
            assert "if (p" not in before and body.count("wait_previous_kernel") == 1, kernel
    assert seen == 5  # two joins, decode, chunk, rotation


@pytest.mark.gpu
@pytest.mark.parametrize("prefix,far", [(0, 300), (0, 9000), (700, 200)])
def test_calls_that_read_what_the_previous_call_wrote(prefix, far):
    """append (rotating q in place, writing the newest keys) and attention right behind it, several steps
    queued without a pause, against the same steps with the device idle between all calls."""
    B, Hq, Hkv, D = 5, 8, 2, 128
    c = Case([1] * B, [far - 37 * b for b in range(B)], Hq=Hq, Hkv=Hkv, D=D, page=64, prefix=prefix, seed=201)
    spec = sa.Rotary([10000.0 ** (-i / 64) for i in range(64)])
    g = torch.Generator().manual_seed(7)
    news = [torch.randn(B, Hq + 2 * Hkv, D, generator=g).bfloat16().cuda() for _ in range(20)]
    pt = c.dev(c.prefix_table)

    def steps(idle):
        cache, batch = c.cache(), c.batch(1)
        q = torch.empty(B, Hq, D, dtype=torch.bfloat16, device="cuda")
        out = []
        for x in news:
            q.copy_(x[:, :Hq])
            if idle:
                torch.cuda.synchronize()
            sa.cache_append(x[:, Hq:Hq + Hkv], x[:, Hq + Hkv:], cache, batch, rotary=spec, pos_offset=prefix, q=q, q_out=q)
            if idle:
                torch.cuda.synchronize()
            p = sa.Pattern(window=1 << 20)
            out += sa.fwd_shared(q, cache, batch, pt, prefix, p) if prefix else sa.fwd_cached(q, cache, batch, p)
            if idle:
                torch.cuda.synchronize()
        torch.cuda.synchronize()
        assert sa.check_device() == sa.SA_OK
        return out

    want = steps(True)
    for _ in range(3):
        for a, b in zip(steps(False), want):
            assert torch.equal(a, b)
