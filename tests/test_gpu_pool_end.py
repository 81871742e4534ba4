"""Pools that end where their allocation ends, with the last block in use and no pool size given: the tensor maps end
there too, and the results are those of pools in the middle of an allocation with the size given."""

import pytest
import torch

from paged_kv_cache_292_gb300 import binding

pytestmark = pytest.mark.gpu

BYTES = 24 << 20  # an allocation of its own, whole 2 MiB pages


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from paged_kv_cache_292_gb300 import build

    build.build()
    binding.load()


def _pool(shape, dtype, seed, at_end):
    """A pool of random values as the last bytes of an allocation, or 4 MiB before them."""
    n = 1
    for x in shape:
        n *= x
    size = n * dtype.itemsize
    gen = torch.Generator().manual_seed(seed)
    arena = torch.empty(BYTES, dtype=torch.uint8, device="cuda")
    end = BYTES - (0 if at_end else 4 << 20)
    pool = arena[end - size : end].view(dtype).view(shape)
    if dtype == torch.uint8:
        pool.copy_(torch.randint(0, 0x70, shape, generator=gen, dtype=torch.uint8))
    else:
        pool.copy_(torch.randn(shape, generator=gen))
    return pool


@pytest.mark.parametrize("Hk, D, bs", [(1, 64, 1), (1, 64, 4), (2, 64, 16), (3, 128, 8), (8, 128, 16), (5, 64, 24)])
@pytest.mark.parametrize("G, Q", [(4, 1), (2, 3), (3, 3), (8, 4)])
@pytest.mark.parametrize("fp8", [False, True])
def test_last_block_of_the_allocation(Hk, D, bs, G, Q, fp8):
    if fp8 and D == 64 and Hk % 2:
        Hk *= 2
    S, nblk = 3, 7
    NB = S * nblk
    dtype = torch.uint8 if fp8 else torch.bfloat16
    gen = torch.Generator().manual_seed(3)
    table = torch.randperm(NB, generator=gen).to(torch.int32)
    last = int((table == NB - 1).nonzero())
    table[last], table[nblk + 3] = int(table[nblk + 3]), NB - 1
    table = table.view(S, nblk).cuda()
    lens = torch.tensor([nblk * bs, nblk * bs - bs // 2, max(Q, nblk * bs - 1)], dtype=torch.int32).cuda()
    q = torch.randn(S, Q, G * Hk, D, generator=gen).to(torch.bfloat16).cuda()
    scales = (0.5, 2.0) if fp8 else ()
    prefix = table[0, :2].contiguous()
    table[:, :2] = prefix  # (the rows' own first blocks go unused)
    outs = []
    for at_end in (True, False):
        k, v = (_pool((NB, bs, Hk, D), dtype, seed, at_end) for seed in (1, 2))
        sizes = (S, Q, G * Hk, Hk, D, bs)
        NBs = 0 if at_end else NB  # no size given: the maps end with the allocation
        lib, stream = binding.load(), torch.cuda.current_stream().cuda_stream
        p = lambda x: x.data_ptr()  # noqa: E731

        def run(name, tables, mid, tail):
            out = torch.full_like(q, float("nan"))
            dtype_arg = () if fp8 else (binding.PA_BF16,)
            rc = getattr(lib, ("pa_decode_fp8_" if fp8 else "pa_decode_") + name)(
                p(out), p(q), p(k), p(v), *(p(t) for t in tables), *sizes, *mid[0], nblk, D**-0.5, *scales, *mid[1],
                stream, *dtype_arg, NBs, None, 0, *tail)
            assert rc == binding.PA_OK, lib.pa_last_error()
            return out

        out = [run("mq", (table, lens), ((), ()), (0, None)),
               run("mod", (table, lens), ((), (0.0, None, 5 * bs, None, None)), (0, None))]
        if bs % 8 == 0:
            out.append(run("prefix", (prefix, table, lens), ((2,), ()), (None,)))
        torch.cuda.synchronize()
        outs.append(out)
    for a, b in zip(*outs):
        assert torch.isfinite(a.float()).all()
        assert torch.equal(a, b)


@pytest.mark.parametrize("name", ["mq", "mod", "prefix"])
@pytest.mark.parametrize("sized", [False, True])
def test_first_call_of_a_thread(name, sized):
    """A caller's workspace, from a host thread that has made no CUDA call before."""
    import threading

    S, Q, Hk, G, D, bs, nblk = 2, 1, 2, 4, 64, 16, 5
    H, NB = G * Hk, S * nblk
    k, v = (_pool((NB, bs, Hk, D), torch.bfloat16, seed, True) for seed in (1, 2))
    table = torch.arange(NB, dtype=torch.int32).view(S, nblk)
    table[1, :2] = table[0, :2].clone()
    prefix, table = table[0, :2].contiguous().cuda(), table.cuda()
    lens = torch.full((S,), nblk * bs, dtype=torch.int32).cuda()
    q = torch.randn(S, Q, H, D).to(torch.bfloat16).cuda()
    out = torch.full_like(q, float("nan"))
    if name == "mq":
        want = binding.decode_multi(q, k, v, table, lens, D**-0.5)
        need, tables, blocks, mods, tail = (binding.pa_decode_mq_workspace_size(S, Q, H, Hk, D), (table, lens), (), (),
                                            (0, None))
    elif name == "mod":
        want = binding.decode_mod(q, k, v, table, lens, D**-0.5, window=50)
        need = binding.pa_decode_mod_workspace_size(S, Q, H, Hk, D, binding.PA_BF16)
        tables, blocks, mods, tail = (table, lens), (), (0.0, None, 50, None, None), (0, None)
    else:
        want = binding.decode_prefix(q, k, v, prefix, table, lens, D**-0.5)
        need = binding.pa_decode_prefix_workspace_size(S, Q, H, Hk, D)
        tables, blocks, mods, tail = (prefix, table, lens), (2,), (), (None,)
    ws = torch.zeros(need, dtype=torch.uint8, device="cuda")
    torch.cuda.synchronize()
    pointers = [x.data_ptr() for x in (out, q, k, v, *tables)]
    lib, said = binding.load(), []

    def call():
        said.append(getattr(lib, "pa_decode_" + name)(*pointers, S, Q, H, Hk, D, bs, *blocks, nblk, D**-0.5, *mods, None,
                                                      binding.PA_BF16, NB if sized else 0, ws.data_ptr(), need, *tail))
        said.append(lib.pa_last_error())

    thread = threading.Thread(target=call)
    thread.start()
    thread.join()
    torch.cuda.synchronize()
    assert said[0] == binding.PA_OK, said
    assert torch.equal(out, want)
