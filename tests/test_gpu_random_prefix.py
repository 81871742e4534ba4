"""Shared-prefix decode against multi-query decode on drawn batches: heads, groups, queries, block sizes, prefixes and
padding rows of every kind, half of them without the pools' size (the library's own view of the memory).

Both sides round their output once (half a step) and weigh the same values: weights in bf16 (2^-8, FP8 pools f16,
2^-11) against 2^-16 (2^-11), with less than 2^-13 from scores and exponentials on either side."""

import random

import pytest
import torch

from paged_kv_cache_292_gb300 import binding

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from paged_kv_cache_292_gb300 import build

    build.build()
    binding.load()


def draw(r):
    while True:
        D, Hk, G, Q = r.choice([64, 128]), r.choice([1, 2, 3, 4, 5, 8, 10]), r.randint(1, 8), r.choice([1, 1, 2, 3, 5, 8])
        fp8 = r.random() < 0.5
        bs, S = r.choice([8, 16, 24, 32, 64, 256]), int(2 ** r.uniform(0, 7))
        P = r.randint(1, max(1, 3000 // bs))
        if G * Q > 32 or (fp8 and D == 64 and Hk % 2):
            continue
        reach = r.choice([Q, Q + 20, 300])
        ctx = [P * bs + r.randint(Q, reach) if r.random() < 0.9 else r.choice([0, r.randint(0, P * bs + Q - 2)])
               for _ in range(S)]
        NB = P + sum(-(-c // bs) for c in ctx) + 2
        if NB * bs * Hk * D <= 1 << 25:
            return D, Hk, G, Q, fp8, bs, S, P, ctx, NB


def one(r, n, sized):
    D, Hk, G, Q, fp8, bs, S, P, ctx, NB = draw(r)
    gen = torch.Generator(device="cuda").manual_seed(n)
    shape = (NB, bs, Hk, D)
    if fp8:  # finite codes below 2
        k, v = (torch.randint(0, 0x40, shape, device="cuda", generator=gen, dtype=torch.uint8)
                | (torch.randint(0, 2, shape, device="cuda", generator=gen, dtype=torch.uint8) << 7) for _ in range(2))
    else:
        k, v = (torch.randn(shape, device="cuda", generator=gen).to(torch.bfloat16) for _ in range(2))
    order = list(range(NB))
    r.shuffle(order)
    prefix, at, rows = order[:P], P, []
    width = max(max(-(-c // bs) for c in ctx), P) + 1
    for c in ctx:
        row = list(prefix) if c >= P * bs + Q - 1 else []
        need = -(-c // bs) - len(row)
        row += order[at : at + need]
        at += need
        rows.append(row + [-1] * (width - len(row)))
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    q = torch.randn(S, Q, G * Hk, D, device="cuda", generator=gen).to(torch.bfloat16)
    table, lens, prefix = i32(rows), i32(ctx), i32(prefix)
    scale = D**-0.5 * r.choice([1, 1, -1, 3])
    scales = (0.7, 1.3) if fp8 else ()
    lib, stream = binding.load(), torch.cuda.current_stream().cuda_stream
    kind = "pa_decode_fp8_" if fp8 else "pa_decode_"
    dtype = () if fp8 else (binding.PA_BF16,)
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    a, b = torch.full_like(q, float("nan")), torch.full_like(q, float("nan"))
    for out, name, tables, blocks, tail in ((a, "prefix", (prefix, table, lens), (P,), ()),
                                            (b, "mq", (table, lens), (), (0,))):
        rc = getattr(lib, kind + name)(
            out.data_ptr(), q.data_ptr(), k.data_ptr(), v.data_ptr(), *(t.data_ptr() for t in tables), S, Q, G * Hk, Hk,
            D, bs, *blocks, width, scale, *scales, stream, *dtype, NB if sized else 0, None, 0, *tail, err.data_ptr())
        assert rc == binding.PA_OK, lib.pa_last_error()
    torch.cuda.synchronize()
    what = f"draw {n}: {dict(D=D, Hk=Hk, G=G, Q=Q, fp8=fp8, bs=bs, S=S, P=P, NB=NB)}"
    assert int(err) == 0, what
    a, b = a.double(), b.double()
    weight = 2 * (2.0**-11 + 2.0**-13) if fp8 else 2.0**-8 + 2.0**-16 + 2 * 2.0**-13
    largest = 1.875 * 1.3 if fp8 else v.abs().max().item()
    assert torch.isfinite(a).all(), what
    assert ((a - b).abs() <= 2.0**-8 * (a.abs() + b.abs()) + weight * largest).all(), what
    # Far below that bound on the whole: rounding errors of either sign.
    assert (a - b).norm() <= 2.0**-7 * b.norm() + 1e-30, what


@pytest.mark.parametrize("sized", [True, False])
@pytest.mark.parametrize("seed", range(4))
def test_drawn_batches(seed, sized):
    r = random.Random(seed)
    for n in range(60):
        one(r, 1000 * seed + n, sized)
